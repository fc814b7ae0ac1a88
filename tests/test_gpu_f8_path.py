"""The 8-bit operators as they are used together: the append into 8-bit
caches, the 8-bit decode step (csa_decode_f8) against the chain of public
calls that it stands for, and the calls that a serving loop makes of them
(captured graphs, other streams, two calls at once, long caches, guarded
buffers, the debug build)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import compressed_sparse_attention_09_b200 as csa
import f8_canary_cases
import f8_ref as ref
from compressed_sparse_attention_09_b200 import synth
from oracle import csa_oracle as orc
from test_gpu_f8 import check_rows, decode_mqa, entries, picked, tc_dims
from test_gpu_parity import check_topk_row, e4m3_codes_f64, gpu_pack

pytestmark = pytest.mark.gpu
DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))


def state(dims, B, cap, pos0, seed):
    """8-bit caches, ring and lengths of B sequences at token pos0."""
    n = B * cap
    Cc = synth.make_normal((n, dims.c), dims, seed + 1).to(DEV)
    Kc = synth.make_normal((n, dims.cI), dims, seed + 2).to(DEV)
    s = dict(Cq=torch.zeros(B, cap, dims.c, dtype=torch.uint8, device=DEV),
             Cs=torch.zeros(B, cap, dtype=torch.uint8, device=DEV),
             Kq=torch.zeros(B, cap, dims.cI, dtype=torch.uint8, device=DEV), Ks=torch.zeros(B, cap, device=DEV),
             ring=synth.make_normal((B, 2 * dims.m, csa.csa_ring_row_elems(dims)), dims, seed + 3).to(DEV),
             clen=torch.full((B,), pos0 // dims.m, dtype=torch.int32, device=DEV))
    csa.csa_quantize_f8(csa.CSA_BF16, Cc, dims.c, n, dims.c, 0, None, 0, s["Cq"], dims.c, s["Cs"], 1)
    csa.csa_quantize_keys_e4m3(Kc, dims.cI, n, dims.cI, s["Kq"], s["Ks"])
    return s


def append(dims, packed, rows, pos, s, cap, B):
    csa.csa_cache_append_f8(dims, packed, rows, pos, s["ring"], s["Cq"], s["Cs"], s["Kq"], s["Ks"], s["clen"], cap, B)


@pytest.mark.parametrize("c,cI,m,pos0", [(512, 128, 4, 6), (64, 64, 2, 0), (1024, 32, 8, 15), (128, 128, 1, 3)])
def test_append_quantises_the_bf16_entry(c, cI, m, pos0):
    """What the 8-bit append stores is the bf16 append's entry, quantised; other rows keep their bytes."""
    dims = csa.Dims(d=64, c=c, m=m, cI=cI, nhI=4, nh=2, dc=64, topk=8, dtype=csa.CSA_BF16)
    B, cap = 5, 12
    packed = gpu_pack(dims, synth.make_weights(dims, 1))
    s = state(dims, B, cap, pos0, 2)
    ring, clen = s["ring"].clone(), s["clen"].clone()
    Cc = torch.zeros(B, cap, c, dtype=torch.bfloat16, device=DEV)
    Kc = torch.zeros(B, cap, cI, dtype=torch.bfloat16, device=DEV)
    want = {k: s[k].clone() for k in ("Cq", "Cs", "Kq", "Ks")}
    for step in range(2 * m + 1):
        rows = synth.make_normal((B, csa.csa_ring_row_elems(dims)), dims, 50 + step).to(DEV)
        pos = torch.full((B,), pos0 + step, dtype=torch.int32, device=DEV)
        append(dims, packed, rows, pos, s, cap, B)
        csa.csa_cache_append(dims, packed, rows, pos, ring, Cc, Kc, clen, cap, B)
        assert csa.csa_get_device_status() == 0
        if (pos0 + step + 1) % m == 0:
            i = (pos0 + step + 1) // m - 1
            cq, cs = ref.quantize(Cc[:, i].double().cpu().numpy(), 0)
            want["Cq"][:, i], want["Cs"][:, i] = torch.as_tensor(cq).to(DEV), torch.as_tensor(cs[:, 0]).to(DEV)
            kq, ks = orc.quantize_e4m3_rows(Kc[:, i].double().cpu().numpy())
            assert np.array_equal(e4m3_codes_f64(s["Kq"][:, i]), kq)
            assert np.array_equal(s["Ks"][:, i].double().cpu().numpy(), ks)
            want["Kq"][:, i], want["Ks"][:, i] = s["Kq"][:, i], s["Ks"][:, i]
    assert torch.equal(s["ring"], ring) and torch.equal(s["clen"], clen)
    for k, v in want.items():
        assert torch.equal(s[k], v), k


def chain(dims, W, packed, h, pos, s, cap, B, idx):
    """The decode step as public calls, given the selection: Y1 / w^I, append, Y2, attention."""
    N1b, N2 = csa.csa_hidden_row_elems(dims), csa.csa_query_row_elems(dims)
    hid = torch.cat([W[k] for k in ("W_aKV", "W_bKV", "W_aZ", "W_bZ", "W_aKV_I", "W_bKV_I", "W_aZ_I", "W_bZ_I", "W_DQ",
                                    "W_w")], 1).t().contiguous().to(DEV)
    qry = torch.cat([W["W_IUQ"], W["W_UQ"]], 1).t().contiguous().to(DEV)

    def weights(w):
        N, K = w.shape
        codes = torch.empty(N, K, dtype=torch.uint8, device=DEV)
        scales = torch.empty(-(-N // 128), -(-K // 128), dtype=torch.uint8, device=DEV)
        csa.csa_quantize_weight_f8(csa.CSA_BF16, w, K, N, K, codes, K, scales, scales.shape[1])
        return codes, scales

    def project(x, ld, K, w, kind):
        codes = torch.empty(B, K, dtype=torch.uint8, device=DEV)
        scales = torch.empty(B, -(-K // 128), dtype=torch.uint8, device=DEV)
        csa.csa_quantize_f8(csa.CSA_BF16, x, ld, B, K, 128, None, 0, codes, K, scales, scales.shape[1])
        N = w[0].shape[0]
        out = torch.empty(B, N, dtype=kind, device=DEV)
        ws = torch.empty(csa.csa_gemm_f8_workspace_bytes(B, N, K), dtype=torch.uint8, device=DEV)
        csa.csa_gemm_f8(csa.CSA_F32 if kind == torch.float32 else csa.CSA_BF16, codes, K, scales, scales.shape[1], w[0], K,
                        w[1], w[1].shape[1], B, N, K, out, N, ws)
        return out

    w1, w2 = weights(hid), weights(qry)
    y1 = project(h, dims.d, dims.d, w1, torch.bfloat16)[:, :N1b].contiguous()
    wI = project(h, dims.d, dims.d, w1, torch.float32)[:, N1b:]
    q0 = 4 * dims.c + 4 * dims.cI
    y2 = project(y1[:, q0:], N1b, dims.dc, w2, torch.bfloat16)
    append(dims, packed, y1[:, :q0].contiguous(), pos, s, cap, B)
    O = torch.empty(B, dims.nh * dims.c, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(csa.csa_mqa_f8_workspace_bytes(dims, B), dtype=torch.uint8, device=DEV)
    csa.csa_decode_mqa_f8(dims, y2[:, dims.nhI * dims.cI:], N2, s["Cq"], s["Cs"], idx, pos, cap, B, O, ws)
    return O, y2, wI


@pytest.mark.parametrize("dims,B,pos0,cap,steps", [
    (csa.Dims(d=256, c=512, m=4, cI=128, nhI=64, nh=64, dc=128, topk=150, dtype=csa.CSA_BF16), 3, 2045, 640, 6),
    (csa.Dims(d=528, c=512, m=4, cI=128, nhI=32, nh=128, dc=144, topk=64, dtype=csa.CSA_BF16), 1, 0, 40, 9),
    (csa.Dims(d=256, c=128, m=2, cI=128, nhI=64, nh=6, dc=128, topk=16, dtype=csa.CSA_BF16), 70, 61, 60, 4),
])
def test_decode_step_is_the_chain_of_its_calls(dims, B, pos0, cap, steps):
    """Several steps across appends: caches, ring and lengths, outputs bit for bit, and the selection a correct top-k
    of the 64-bit scores of the step's own q^I and w^I (tests/parity.py's rule with eq. (8)'s fp32 error)."""
    W = synth.make_weights(dims, 21)
    packed = gpu_pack(dims, W)
    packed8 = torch.empty(csa.csa_packed_weights_f8_bytes(dims), dtype=torch.uint8, device=DEV)
    csa.csa_pack_weights_f8(dims, packed, packed8)
    s = state(dims, B, cap, pos0, 30)
    t = {k: v.clone() for k, v in s.items()}
    ws = torch.empty(csa.csa_decode_f8_workspace_bytes(dims, B, cap), dtype=torch.uint8, device=DEV)
    for step in range(steps):
        h = synth.make_normal((B, dims.d), dims, 100 + step).to(DEV)
        pos = torch.full((B,), pos0 + step, dtype=torch.int32, device=DEV)
        O = torch.empty(B, dims.nh * dims.c, dtype=torch.bfloat16, device=DEV)
        idx = torch.full((B, dims.topk), -9, dtype=torch.int32, device=DEV)
        csa.csa_decode_f8(dims, packed, packed8, h, pos, s["ring"], s["Cq"], s["Cs"], s["Kq"], s["Ks"], s["clen"], cap, B, O,
                          idx, ws)
        assert csa.csa_get_device_status() == 0
        want, y2, wI = chain(dims, W, packed, h, pos, t, cap, B, idx)
        assert csa.csa_get_device_status() == 0
        for k in s:
            assert torch.equal(s[k], t[k]), (step, k)
        assert torch.equal(O, want), step
        avail = (pos0 + step) // dims.m
        for b in range(min(B, 4)):
            qI = y2[b, :dims.nhI * dims.cI].double().cpu().numpy().reshape(dims.nhI, dims.cI)
            K = e4m3_codes_f64(s["Kq"][b, :avail]) * s["Ks"][b, :avail].double().cpu().numpy()[:, None]
            w = wI[b].double().cpu().numpy()
            scores = (w[:, None] * np.maximum(qI @ K.T, 0)).sum(0)
            delta = (dims.cI + dims.nhI + 2) * 2.0 ** -23 * (np.abs(w)[:, None] * (np.abs(qI) @ np.abs(K).T)).sum(0)
            delta = delta + 2.0 ** -11 * 2.0 ** -14 * np.abs(w).sum() * np.abs(K).sum(1)   # q^I in fp16: subnormal below 2^-14
            check_topk_row(idx[b].cpu().numpy(), scores, dims.topk, delta)


def test_decode_step_approximates_the_bf16_step():
    """Against csa_decode on the same state: E4M3 weights, activations and entries (rounding within 2^-4 relative) leave
    the output's direction: with every entry selected, a relative 2-norm below 0.2 (two chained products of relative
    error 2^-4 / sqrt(3) per factor: sqrt(2) * 3.6 % * sqrt(2) each, entries 3.6 %: 0.11)."""
    dims = csa.Dims(d=512, c=512, m=4, cI=128, nhI=64, nh=64, dc=256, topk=100, dtype=csa.CSA_BF16)
    B, cap, pos0 = 4, 100, 400
    W = synth.make_weights(dims, 5)
    packed = gpu_pack(dims, W)
    packed8 = torch.empty(csa.csa_packed_weights_f8_bytes(dims), dtype=torch.uint8, device=DEV)
    csa.csa_pack_weights_f8(dims, packed, packed8)
    s = state(dims, B, cap, pos0, 6)
    Cc = synth.make_normal((B * cap, dims.c), dims, 7).to(DEV)
    Kc = synth.make_normal((B * cap, dims.cI), dims, 8).to(DEV)
    ring, clen = s["ring"].clone(), s["clen"].clone()
    h = synth.make_normal((B, dims.d), dims, 9).to(DEV)
    pos = torch.full((B,), pos0, dtype=torch.int32, device=DEV)
    O8, O16 = (torch.empty(B, dims.nh * dims.c, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.empty(csa.csa_decode_f8_workspace_bytes(dims, B, cap), dtype=torch.uint8, device=DEV)
    csa.csa_decode_f8(dims, packed, packed8, h, pos, s["ring"], s["Cq"], s["Cs"], s["Kq"], s["Ks"], s["clen"], cap, B, O8,
                      None, ws)
    csa.csa_decode(dims, packed, h, pos, ring, Cc, Kc, clen, cap, B, O16, None, ws)
    assert csa.csa_get_device_status() == 0
    # (state() draws its bf16 caches with seeds 7 and 8 as well)
    d = (O8.double() - O16.double()).norm() / O16.double().norm()
    assert d < 0.2, float(d)


# ---------------------------------------------------------------- graphs, streams, two calls at once
def mqa_call(dims, B, cap, seed):
    rng = np.random.default_rng(seed)
    codes, scales = entries(rng, B * cap, 512)
    q = torch.as_tensor(rng.standard_normal((B, dims.nh * 512)), dtype=torch.float32).to(torch.bfloat16).to(DEV)
    idx = picked(rng, B, dims.topk, [cap] * B).to(DEV)
    pos = torch.full((B,), 4 * cap, dtype=torch.int32, device=DEV)
    out = torch.zeros(B, dims.nh * 512, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(csa.csa_mqa_f8_workspace_bytes(dims, B), dtype=torch.uint8, device=DEV)
    call = lambda stream=None: csa.csa_decode_mqa_f8(dims, q, dims.nh * 512, codes, scales, idx, pos, cap, B, out, ws, stream)  # noqa: E731
    return call, dict(q=q, codes=codes, scales=scales, idx=idx, out=out)


def gemm_call(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a, b = (torch.randint(0, 0x60, (n, K), generator=g).to(torch.uint8).to(DEV) for n in (M, N))
    sa = torch.randint(120, 130, (M, -(-K // 128)), generator=g).to(torch.uint8).to(DEV)
    sb = torch.randint(120, 130, (-(-N // 128), -(-K // 128)), generator=g).to(torch.uint8).to(DEV)
    out = torch.zeros(M, N, device=DEV)
    ws = torch.empty(csa.csa_gemm_f8_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    call = lambda stream=None: csa.csa_gemm_f8(csa.CSA_F32, a, K, sa, sa.shape[1], b, K, sb, sb.shape[1], M, N, K, out, N, ws, stream)  # noqa: E731
    return call, dict(a=a, b=b, sa=sa, sb=sb, out=out)


def test_captured_and_replayed_with_new_inputs():
    """Both operators that use a workspace (split attention and its join, K-split product and its reduction) captured
    into two graphs; replays after the inputs changed give what plain calls give."""
    dims = tc_dims(128, 300)
    calls = [mqa_call(dims, 1, 400, 1), gemm_call(7, 300, 1024, 2)]
    st = torch.cuda.Stream()
    graphs = []
    for call, _ in calls:
        with torch.cuda.stream(st):
            call()
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call()
            graphs.append(g)
    for k in range(3):
        calls[0][1]["q"].mul_(0.5 + k)
        calls[1][1]["sa"].add_(1)
        for g in (graphs if k % 2 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        got = [t["out"].clone() for _, t in calls]
        for call, t in calls:
            t["out"].zero_()
            call()
        torch.cuda.synchronize()
        assert csa.csa_get_device_status() == 0
        for (_, t), v in zip(calls, got):
            assert torch.equal(t["out"], v) and v.abs().sum() > 0


def test_two_calls_at_once_on_two_streams():
    dims = tc_dims(64, 500)
    calls = [mqa_call(dims, 2, 600, 3), mqa_call(dims, 30, 600, 4), gemm_call(20, 400, 2048, 5), gemm_call(500, 700, 512, 6)]
    want = []
    for call, t in calls:
        call()
        torch.cuda.synchronize()
        want.append(t["out"].clone())
        t["out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (call, _), st in zip(calls, streams):
            call(st)
    torch.cuda.synchronize()
    assert csa.csa_get_device_status() == 0
    for (_, t), v in zip(calls, want):
        assert torch.equal(t["out"], v)


def test_calls_follow_their_stream_order():
    """Write, read back and attention queued on a side stream behind a slow producer see its results."""
    st = torch.cuda.Stream()
    n, w = 5000, 512
    x = torch.randn(n, w, device=DEV)
    codes = torch.zeros(n, w, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, 1, dtype=torch.uint8, device=DEV)
    y = torch.zeros(n, w, dtype=torch.bfloat16, device=DEV)
    src = torch.zeros(n, w, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(5):
            big = big @ big * 1e-2
        src.copy_(x.to(torch.bfloat16))
        csa.csa_quantize_f8(csa.CSA_BF16, src, w, n, w, 0, None, 0, codes, w, scales, 1)
        csa.csa_dequantize_f8(csa.CSA_BF16, codes, w, scales, 1, n, w, 0, None, n, y, w)
        z = y.float() * 2
    st.synchronize()
    c, s = ref.quantize(x[:40].to(torch.bfloat16).double().cpu().numpy(), 0)
    assert np.array_equal(codes[:40].cpu().numpy(), c) and np.array_equal(scales[:40].cpu().numpy(), s)
    assert torch.equal(z, y.float() * 2) and (y.float() - x).norm() < 0.05 * x.norm()


# ---------------------------------------------------------------- far offsets
def test_cache_offsets_beyond_32_bits():
    """Rows whose byte offset passes 2^32, written, read back and attended to."""
    cap, w = 4_300_000, 512                      # two sequences: 4.4 GB of codes
    codes = torch.zeros(2 * cap, w, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(2 * cap, 1, dtype=torch.uint8, device=DEV)
    far = torch.tensor([2 * cap - 1, 2 * cap - 70, cap + 4_200_000, cap + 5], dtype=torch.int32)
    assert int(far[0]) * w > 2 ** 31 and int(far[2]) * w > 2 ** 32
    x = torch.randn(4, w).to(torch.bfloat16)
    csa.csa_quantize_f8(csa.CSA_BF16, x.to(DEV), w, 4, w, 0, far.to(DEV), 2 * cap, codes, w, scales, 1)
    c, s = ref.quantize(x.double().numpy(), 0)
    assert np.array_equal(codes[far.long().to(DEV)].cpu().numpy(), c)
    y = torch.empty(4, w, device=DEV)
    csa.csa_dequantize_f8(csa.CSA_F32, codes, w, scales, 1, 2 * cap, w, 0, far.to(DEV), 4, y, w)
    assert torch.equal(y.cpu().double(), ref.decode(torch.as_tensor(c), torch.as_tensor(s), 0))
    dims = tc_dims(64, 70)
    idx = torch.full((2, 70), -1, dtype=torch.int32)
    idx[1, :4] = far - cap
    idx[0, 3] = cap - 1
    q, _, _, out = decode_mqa(dims, 2, cap, [cap, cap], idx, 3, codes=codes, scales=scales.view(-1))
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales.view(-1), idx, [0, cap], [cap, cap], out)


# ---------------------------------------------------------------- guarded buffers, debug build
@pytest.fixture(scope="module")
def release():
    return f8_canary_cases.run_all()


def clean(res):
    for k, v in res.items():
        if k.endswith("/status"):
            assert int(v[0]) == 0, k
        if k.endswith("/pads_intact"):
            assert bool(v[0]), k


def test_guard_bytes_stay_intact(release):
    clean(release)


def test_debug_build_gives_the_same_bytes(release, tmp_path):
    path = str(tmp_path / "debug.npz")
    r = subprocess.run([sys.executable, os.path.join(HERE, "f8_canary_cases.py"), path], env=dict(os.environ, CSA_DEBUG="1"),
                       cwd=HERE, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    debug = dict(np.load(path))
    clean(debug)
    assert set(debug) == set(release)
    for k, v in release.items():
        assert np.array_equal(debug[k], v), k
