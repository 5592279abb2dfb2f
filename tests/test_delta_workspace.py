"""qsa_delta_prompt_workspace_bytes is what the header says, and no more than the chunks that a step can have."""
import os
import re

import pytest

from test_linear_abi import lib  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qsa.h")


@pytest.mark.parametrize("n_tok,n_seq,n_k,n_v,cut", [(33, 1, 16, 32, False), (33, 2, 16, 32, False), (2512, 512, 16, 32, False),
                                                     (12 * 4096, 12, 16, 32, False), (8192, 1, 16, 32, True), (4096, 2, 1, 2, True)])
def test_the_header_s_formula(lib, n_tok, n_seq, n_k, n_v, cut):  # noqa: F811
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER, encoding="utf-8").read())
    per_k, per_v, each = (int(x.replace(",", "")) for x in re.search(
        r"([\d,]+) n_k \+ ([\d,]+) n_v bytes for each of n_tok / 64 \+ n_seq chunks, or for each of n_tok / 32 in a step of several "
        r"sequences if those are fewer; .*?([\d,]+) n_v bytes a token and 1 MB n_seq n_v more", text).groups())
    chunks = n_tok // 64 + n_seq if n_seq == 1 else min(n_tok // 64 + n_seq, n_tok // 32)
    want = chunks * (per_k * n_k + per_v * n_v) + (n_tok * each * n_v + (n_seq * n_v << 20) if cut else 0)
    assert 0 <= lib.qsa_delta_prompt_workspace_bytes(n_tok, n_seq, n_k, n_v) - want <= 256


def test_steps_without_chunks_need_none(lib):  # noqa: F811
    for n_tok, n_seq in ((0, 3), (1, 1), (2, 1), (32, 1), (32, 32)):
        assert lib.qsa_delta_prompt_workspace_bytes(n_tok, n_seq, 16, 32) == 256


def test_short_sequences_need_little(lib):  # noqa: F811
    """512 sequences' single tokens beside a prompt of 2,000."""
    assert lib.qsa_delta_prompt_workspace_bytes(2512, 512, 16, 32) < 110 << 20
