"""The attention over 8-bit entries at the ends of the scales' range: zero
entries (scale byte 0), whole parts of them, and scales near 2^-127 and 2^120,
for rows that are split over their parts and for the same rows unsplit."""
import math

import numpy as np
import pytest
import torch

import compressed_sparse_attention_09_b200 as csa
import f8_ref as ref
from test_gpu_f8 import BF16, DEV, F32, decode_mqa, entries, tc_dims

pytestmark = pytest.mark.gpu
PART = 64   # entries of a part: a row that is split gives each split whole parts


def check(dims, q, codes, scales, out, cap, rows):
    """Rows that select all of their `cap` entries, against the 64-bit definition."""
    assert csa.csa_get_device_status() == 0
    for r in rows:
        sel = r * cap + torch.arange(cap, device=DEV)
        want, bound = ref.mqa(q[r].double().view(dims.nh, 512), codes, scales, sel, BF16)
        err = (out[r].double().view(dims.nh, 512) - want).abs()
        assert (err <= bound).all(), (r, float((err / bound).nan_to_num(math.inf).max()))


def run(kind, nh, cap, B, change, positive=False):
    """B rows over `cap` entries each, all selected; change(codes, scales, row's first entry) sets the entries apart."""
    rng = np.random.default_rng(len(kind) + nh + cap)
    dims = tc_dims(nh, cap)
    assert (csa.csa_mqa_f8_workspace_bytes(dims, B) > 0) == (B == 1)   # one row is split, many are not
    codes, scales = entries(rng, cap, 512)
    change(codes, scales)
    codes, scales = codes.repeat(B, 1), scales.repeat(B)
    q = rng.standard_normal((1, nh * 512))
    q = torch.as_tensor(np.abs(q) if positive else q, dtype=F32).to(BF16).repeat(B, 1).to(DEV)
    idx = torch.arange(cap, dtype=torch.int32).repeat(B, 1)
    q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 1, codes=codes, scales=scales, q=q)
    check(dims, q, codes, scales, out, cap, sorted({0, B // 2, B - 1}))


def zero(codes, scales, at):
    codes[at], scales[at] = 0, 0


KINDS = {
    "first part zero": lambda c, s: zero(c, s, slice(0, PART)),
    "last part zero": lambda c, s: zero(c, s, slice((len(s) - 1) // PART * PART, None)),
    "middle and first parts zero": lambda c, s: [zero(c, s, slice(p, p + PART)) for p in (0, len(s) // 2 // PART * PART)],
    "all zero": lambda c, s: zero(c, s, slice(None)),
    "all but one zero": lambda c, s: [zero(c, s, slice(0, 70)), zero(c, s, slice(71, None))],
    "a part of byte 0, codes not zero": lambda c, s: s[:PART].fill_(0),
    "a part of bytes 1 to 3": lambda c, s: s[:PART].copy_(torch.arange(PART) % 3 + 1),
}


@pytest.mark.parametrize("B", [1, 160])
@pytest.mark.parametrize("nh,cap", [(64, 128), (128, 700)])
@pytest.mark.parametrize("kind", KINDS)
def test_zero_entries_and_tiny_scales_keep_their_share(kind, nh, cap, B):
    """A part whose entries are zero, or next to it, counts in the normaliser, whichever split it falls into."""
    run(kind, nh, cap, B, KINDS[kind])


@pytest.mark.parametrize("B", [1, 160])
def test_zero_entries_beside_scores_far_below_theirs(B):
    """In one part zero entries (score 0) and entries with scores of about -180 (base 2)."""
    def change(codes, scales):
        zero(codes, scales, slice(0, PART, 2))
        codes[1:PART:2], scales[1:PART:2] = 0xFE, 121        # -448 * 2^-6 in every channel, against queries above zero
    run("far", 64, 192, B, change, positive=True)
