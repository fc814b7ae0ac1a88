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


def check(dims, q, codes, scales, out, cap, rows, one_channel=False):
    """Rows that select all of their `cap` entries, against the 64-bit definition and ref.mqa's bound, but for two terms.
    Weights are relative to a maximum that counts no scale below 2^-118, so the error of 2^-16 of the largest weight is
    of no less than the largest probability times 2^-118.  And where a head's query is one channel (its 8 significant
    bits are held) and zeros, the scores have the errors of fp32 alone."""
    assert csa.csa_get_device_status() == 0
    table = torch.as_tensor(ref.TABLE, device=DEV)
    for r in rows:
        sel = r * cap + torch.arange(cap, device=DEV)
        x = q[r].double().view(dims.nh, 512)
        raw, sc = table[codes[sel].long()], torch.exp2(scales[sel].double() - 127)
        e = raw * sc[:, None]
        s = x @ e.t() / math.sqrt(512)
        p = torch.softmax(s, 1)
        if one_channel:
            want = p @ e
            dp = p * torch.expm1(2 * (516 * 2.0 ** -23 * s.abs() + 2.0 ** -20 * (1 + s.abs())))
            bound = ((2.0 ** -7 + 2.0 ** -10) * p + dp) @ e.abs() + dp.sum(1, keepdim=True) * want.abs()
            bound = bound + 2.0 ** -16 * (p * sc).amax(1, keepdim=True) * raw.abs().sum(0)[None]
            bound = bound + ref.half_step(BF16) * (want.abs() + bound) + 1e-37
        else:
            want, bound = ref.mqa(x, codes, scales, sel, BF16)
        bound = bound + 2.0 ** (-16 - 118) * p.amax(1, keepdim=True) * raw.abs().sum(0)
        err = (out[r].double().view(dims.nh, 512) - want).abs()
        assert (err <= bound).all(), (r, float((err / bound).nan_to_num(math.inf).max()))


def run(kind, nh, cap, B, change, positive=False):
    """B rows over `cap` entries each, all selected; change(codes, scales, row's first entry) sets the entries apart."""
    rng = np.random.default_rng(len(kind) + nh + cap)
    dims = tc_dims(nh, cap)
    if nh % 64 == 0:   # tensor cores: one row is split, many are not
        assert (csa.csa_mqa_f8_workspace_bytes(dims, B) > 0) == (B == 1)
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
@pytest.mark.parametrize("nh,cap", [(64, 128), (128, 700), (20, 130)])
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


@pytest.mark.parametrize("nh,B", [(64, 1), (64, 160), (20, 3)])
@pytest.mark.parametrize("low,high", [(0, 0), (0, 1), (1, 1), (1, 5), (0, 20), (9, 9)])
def test_nothing_but_tiny_scales(low, high, nh, B):
    """Entries of 128 to 448 times 2^-127 .. 2^-107: outputs of 1e-36 and more, which bf16 holds as normal numbers."""
    def change(codes, scales):
        codes[:] = codes % 15 + 0x70
        scales[:] = low + scales % (high - low + 1)
    run("tiny", nh, 192, B, change)


@pytest.mark.parametrize("B", [1, 160])
@pytest.mark.parametrize("byte", [240, 244, 247])
def test_huge_scales_keep_the_weights_of_lower_scores(byte, B):
    """Entries of 2^(byte - 122) and one score some 10 to 20 (base 2) above all others, whose weights add up to up to a
    tenth of the whole."""
    rng = np.random.default_rng(byte)
    cap, dims = 128, tc_dims(64, 128)
    codes = torch.as_tensor(rng.integers(0x60, 0x69, (cap, 512)).astype(np.uint8))
    codes[:, 0] = 0x44                                        # 3 in the only channel that the queries see,
    codes[0, 0] = 0x50                                        # 8 in the first entry
    q = torch.zeros(64, 512, dtype=F32)
    q[:, 0] = 2.0 ** (132 - byte) * (1 + torch.arange(64) / 64)   # scores 2.04 (1 + h / 64) times the code
    q = q.to(BF16).view(1, -1).repeat(B, 1).to(DEV)
    idx = torch.arange(cap, dtype=torch.int32).repeat(B, 1)
    q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 1, codes=codes.repeat(B, 1).to(DEV), q=q,
                                       scales=torch.full((B * cap,), byte, dtype=torch.uint8, device=DEV))
    check(dims, q, codes, scales, out, cap, sorted({0, B - 1}), one_channel=True)
