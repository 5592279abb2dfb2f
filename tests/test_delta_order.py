"""Products on the tensor cores are ordered among themselves only where they share accumulator and shape.  delta_chunk_kernel's
source: every accumulator has one shape, and what one product reads and another writes has a wait between them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_selected_cell_gb300", "csrc")
CODE = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "delta_prompt.cu"), encoding="utf-8").read())
ROLE = re.search(r"void product_role\(.*?\n}\n", CODE, re.S).group(0)
COLUMNS = {n: int(v) for n, v in re.findall(r"(kTm\w+) = (\d+)", CODE)}
WIDTH = {"id64": 64, "id32": 32, "idD": 128}


def products():
    """(accumulator's first column, its width, operand's name) of every product."""
    found = re.findall(r"product\(c\.tmem \+ (kTm\w+)(?: \+ (\d+))?,\s*(.*?), (id\w*),", ROLE, re.S)
    assert len(found) == ROLE.count("product(c.") and len(found) >= 8
    return [(COLUMNS[name] + int(more or 0), WIDTH[shape], rest) for name, more, rest, shape in found]


def test_an_accumulator_has_one_shape():
    spans = {(at, width) for at, width, _ in products()}
    assert all(a == b or a[0] + a[1] <= b[0] or b[0] + b[1] <= a[0] for a in spans for b in spans), spans
    assert not re.search(r"\bid\w* [-+]", ROLE)


def test_keys_wait_for_the_outputs_before():
    """S K^T's columns hold V' P^T's operand of the chunk before."""
    assert COLUMNS["kTmKs"] < COLUMNS["kTmH"] + 64 and COLUMNS["kTmH"] < COLUMNS["kTmKs"] + 64
    assert re.search(r"i > 0 && !\(ok = wait\(c, BAR_O, par \^ 1\)\)", ROLE).start() < ROLE.index("product(c.tmem + kTmKs")


def test_values_wait_for_the_outputs_before():
    """V' and V' P^T share their columns; so do S Q^T of a chunk and of the next."""
    assert COLUMNS["kTmV"] == COLUMNS["kTmPv"]
    assert re.search(r"i > 0 && !\(ok = wait\(c, BAR_OFREE, par \^ 1\)\)", ROLE).start() < ROLE.index("product(c.tmem + kTmV")
