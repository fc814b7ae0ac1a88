"""What is measured of the 8-bit operators: the cases, their inputs, their plain form and the calls.

The operators keep values as E4M3 codes with one power-of-two scale for each block of a row: a code c under the
scale byte b stands for c * 2^(b - 127).  Four of them are measured:

  write   rows to codes and scales, put into the rows of a cache (or of an activation matrix) that `slots` names
  read    rows of such a cache, named by `rows`, back to bf16 or fp32
  gemm    D = A . B^T of two such matrices: A with a scale for 1 x 128 values, B for 128 x 128
  mqa     the shared-key-value attention of each query row over the cache entries that its index row selects

`run` gives each in its plain form (32-bit torch operations) or, where `own` is true, through the framework's calls.
`exact` gives them in 64 bits, from their definitions.
"""
import math

import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    """Twelve cases: the sizes are those of the repository's prefill, ragged, long and decode workloads."""
    return [
        # a decode step's new entries, one for each of 64 sequences: launch latency is all there is
        dict(name="write_64", op="write", n=64, w=512, block=0, dtype="bf16", slots=4096),
        # the entries of a prefill of 131072 tokens (m = 4), scattered to the rows of a cache
        dict(name="write_32768", op="write", n=32768, w=512, block=0, dtype="bf16", slots=40000),
        # the hidden rows of a prefill of 8192 tokens, quantised for the 8-bit projection
        dict(name="activations_8192", op="write", n=8192, w=4096, block=128, dtype="bf16", slots=0),
        # the entries that one query selects, read back
        dict(name="read_2048", op="read", n=2048, w=512, block=0, dtype="bf16", slots=16448),
        # the entries that 64 decoding sequences select (k = 2048 each), in fp32
        dict(name="read_131072", op="read", n=131072, w=512, block=0, dtype="f32", slots=262144),
        # the hidden-side projection of a decode step (64 rows: the weights are the traffic)
        dict(name="gemm_hidden_64", op="gemm", M=64, N=4160, K=4096, dtype="bf16"),
        # the query-side projection of a decode step with 128 heads
        dict(name="gemm_query_64", op="gemm", M=64, N=73728, K=1536, dtype="bf16"),
        # the hidden-side projection of an odd number of prefill rows, kept in fp32
        dict(name="gemm_hidden_1001", op="gemm", M=1001, N=4160, K=4096, dtype="f32"),
        # the query-side projection of a prefill of 8192 tokens: the largest product of the forward
        dict(name="gemm_query_8192", op="gemm", M=8192, N=40960, K=1536, dtype="bf16"),
        # one decoding sequence over 16384 entries, 128 heads, 2048 selected: too few rows to fill the GPU by rows
        dict(name="mqa_decode_1", op="mqa", rows=1, nh=128, k=2048, avail=16384, decode=True),
        # 64 decoding sequences of the same kind
        dict(name="mqa_decode_64", op="mqa", rows=64, nh=128, k=2048, avail=16384, decode=True),
        # a prefill of 8192 tokens in three packed sequences, 64 heads, 512 selected; early rows select fewer or none
        dict(name="mqa_prefill_8192", op="mqa", rows=8192, nh=64, k=512, avail=0, decode=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: sizes over their logarithm, widths and depths in steps of 16, odd counts of rows."""
    op = rng.choice(("write", "read", "gemm", "mqa"))
    if op in ("write", "read"):
        w = 16 * _log(rng, 4, 256)
        n = _log(rng, 1, min(65536, (1 << 25) // w))
        block = rng.choice((0, 128)) if w <= 1024 else 128
        slots = 0 if op == "write" and rng.random() < 0.4 else n + rng.randrange(1, 5000)
        return dict(op=op, n=n, w=w, block=block, dtype=rng.choice(("bf16", "f32")), slots=slots)
    if op == "gemm":
        M, N, K = _log(rng, 1, 8192), _log(rng, 64, 40960), 16 * _log(rng, 8, 256)
        while M * N * K > 1 << 37 or M * N > 1 << 27:
            M, N = max(1, M // 2), max(64, N // 2 + 1)
        return dict(op="gemm", M=M, N=N, K=K, dtype=rng.choice(("bf16", "f32")))
    decode = rng.random() < 0.6
    rows = _log(rng, 1, 96) if decode else _log(rng, 16, 4000)
    avail = _log(rng, 1, 16384) if decode else 0
    return dict(op="mqa", rows=rows, nh=rng.choice((64, 128)), k=_log(rng, 1, 2048) if decode else _log(rng, 8, 512), avail=avail, decode=decode)


def _lens(rows):
    """Three packed sequences (one where there are few rows), of unequal and odd lengths."""
    if rows < 64:
        return [rows]
    a, b = rows * 3 // 8 + 1, rows // 5
    return [a, b, rows - a - b]


def work(case):
    if case["op"] in ("write", "read"):
        n, w = case["n"], case["w"]
        es = 2 if case["dtype"] == "bf16" else 4
        scales = n * (1 if case["block"] == 0 else -(-w // 128))
        index = 4 * n if case["slots"] else 0
        return {"bytes": n * w * (es + 1) + scales + index, "flops": 0}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * K + N * K + M * kb + -(-N // 128) * kb + M * N * es, "flops": 2 * M * N * K}
    rows, nh, k = case["rows"], case["nh"], case["k"]
    if case["decode"]:
        sel = rows * min(k, case["avail"])
        entries = sel
    else:
        sel = sum(min(k, t // 4) for n in _lens(rows) for t in range(n))
        entries = sum(n // 4 for n in _lens(rows))
    return {"bytes": rows * nh * 512 * 4 + rows * k * 4 + entries * 513, "flops": 4 * 512 * nh * sel}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _encode(x, block):
    """Rows in fp32 to (codes as float8, scale bytes): the inputs of the operators that read codes."""
    n, w = x.shape
    kb = -(-w // block)
    pad = torch.nn.functional.pad(x, (0, kb * block - w)).view(n, kb, block)
    mant, ex = torch.frexp(pad.abs().amax(-1))
    byte = torch.where(mant > 0, (ex - 9 + (mant > 0.875) + 127).clamp(0, 254), 0)
    y = torch.ldexp(pad, 127 - byte[..., None]).view(n, kb * block)[:, :w]
    return y.to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _pick(g, rows, visible, k):
    """Index rows: for each row up to k distinct blocks below visible[row], ascending, then -1."""
    n = int(visible.max())
    if n == 0:
        return torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
    key = torch.rand(rows, n, generator=g, device=DEV)
    key = torch.where(torch.arange(n, device=DEV) < visible[:, None], key, -1.0)
    val, at = torch.topk(key, min(k, n), dim=1)
    at = torch.where(val >= 0, at, 1 << 30).sort(1).values
    at = torch.where(at < 1 << 30, at, -1).to(torch.int32)
    return torch.nn.functional.pad(at, (0, k - at.shape[1]), value=-1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "write":
        n, w = case["n"], case["w"]
        x = _normal(g, n, w) * torch.exp2(3 * _normal(g, n, 1))      # rows of unequal magnitude
        s["x"] = x.to(TYPES[case["dtype"]])
        rows = case["slots"] or n
        s["at"] = torch.randperm(rows, generator=g, device=DEV)[:n].to(torch.int32) if case["slots"] else None
        s["codes"] = torch.zeros(rows, w, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(rows, 1 if case["block"] == 0 else -(-w // 128), dtype=torch.uint8, device=DEV)
    elif case["op"] == "read":
        n, w, rows = case["n"], case["w"], case["slots"]
        codes, s["scales"] = _encode(_normal(g, rows, w) * torch.exp2(3 * _normal(g, rows, 1)), case["block"] or w)
        s["codes"] = codes.view(torch.uint8)
        s["at"] = torch.randint(0, rows, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["at"][torch.rand(n, generator=g, device=DEV) < 0.01] = -1   # empty places of a selection
        s["out"] = torch.empty(n, w, dtype=TYPES[case["dtype"]], device=DEV)
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a, s["sa"] = _encode(_normal(g, M, K) * torch.exp2(_normal(g, M, 1)), 128)
        nb, kb = -(-N // 128), -(-K // 128)
        byte = torch.randint(110, 119, (nb, kb), generator=g, device=DEV)   # weights of about 1 / sqrt(K)
        b = torch.randn(N, K, generator=g, device=DEV, dtype=torch.bfloat16) * 64
        s["a"], s["b"], s["sb"] = a.view(torch.uint8), b.to(torch.float8_e4m3fn).view(torch.uint8), byte.to(torch.uint8)
        s["out"] = torch.empty(M, N, dtype=TYPES[case["dtype"]], device=DEV)
    else:
        rows, nh, k = case["rows"], case["nh"], case["k"]
        s["q"] = torch.randn(rows, nh * 512, generator=g, device=DEV, dtype=torch.bfloat16)
        if case["decode"]:
            cap = case["avail"] + 3
            visible = torch.full((rows,), case["avail"], device=DEV)
            s["pos"] = torch.full((rows,), 4 * case["avail"] + 1, dtype=torch.int32, device=DEV)
            s["cap"], s["base"] = cap, torch.arange(rows, device=DEV) * cap
            total = rows * cap
        else:
            lens = _lens(rows)
            cu = [0] + [sum(lens[: i + 1]) for i in range(len(lens))]
            cb = [0] + [sum(n // 4 for n in lens[: i + 1]) for i in range(len(lens))]
            visible = torch.cat([torch.arange(n, device=DEV) // 4 for n in lens])
            s["base"] = torch.cat([torch.full((n,), cb[i], device=DEV) for i, n in enumerate(lens)])
            s["cu"], s["cb"] = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (cu, cb))
            total = cb[-1]
        s["codes"] = torch.empty(total, 512, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(total, dtype=torch.uint8, device=DEV)
        for i in range(0, total, 1 << 18):
            n = min(1 << 18, total - i)
            codes, scales = _encode(_normal(g, n, 512) * torch.exp2(0.5 * _normal(g, n, 1)), 512)
            s["codes"][i: i + n], s["scales"][i: i + n] = codes.view(torch.uint8), scales[:, 0]
        s["idx"] = _pick(g, rows, visible, k)
        s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"write": _write, "read": _read, "gemm": _gemm, "mqa": _mqa}[s["op"]](s)


def _value(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _scale(byte):
    return torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127)


def _write(s):
    x = s["x"].float()
    n, w = x.shape
    block = s["block"] or w
    kb = -(-w // block)
    pad = torch.nn.functional.pad(x, (0, kb * block - w)).view(n, kb, block)
    mant, ex = torch.frexp(pad.abs().amax(-1))
    byte = torch.where(mant > 0, (ex - 9 + (mant > 0.875) + 127).clamp(0, 254), 0)
    y = (pad * _scale(254 - byte)[..., None]).view(n, kb * block)[:, :w]
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    at = slice(0, n) if s["at"] is None else s["at"].long()
    s["codes"][at] = codes
    s["scales"][at] = byte.to(torch.uint8)
    return s["codes"].view(torch.float8_e4m3fn), s["scales"]


def _read(s):
    at = s["at"].long()
    some = (at >= 0)[:, None]
    at = at.clamp(min=0)
    block = s["block"] or s["w"]
    scale = _scale(s["scales"][at]).repeat_interleave(block, 1)[:, : s["w"]]
    return torch.where(some, _value(s["codes"][at]) * scale, 0.0).to(s["out"].dtype)


def _gemm(s):
    a = _value(s["a"]) * _scale(s["sa"]).repeat_interleave(128, 1)[:, : s["K"]]
    b = _value(s["b"]) * _scale(s["sb"]).repeat_interleave(128, 0)[: s["N"]].repeat_interleave(128, 1)[:, : s["K"]]
    return torch.matmul(a, b.t()).to(s["out"].dtype)


def _mqa(s):
    rows, nh = s["rows"], s["nh"]
    some = s["idx"] >= 0
    at = s["base"][:, None] + s["idx"].clamp(min=0).long()
    e = _value(s["codes"][at]) * _scale(s["scales"][at])[..., None]
    q = s["q"].view(rows, nh, 512).float()
    t = torch.matmul(q, e.transpose(1, 2)) * 512 ** -0.5
    t = torch.where(some[:, None], t, -math.inf)
    p = torch.exp(t - t.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(p, e) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.to(torch.bfloat16).view(rows, nh * 512)


def _own(s):
    import compressed_sparse_attention_09_b200 as csa
    kind = {torch.bfloat16: csa.CSA_BF16, torch.float32: csa.CSA_F32}
    if s["op"] == "write":
        csa.csa_quantize_f8(kind[s["x"].dtype], s["x"], s["w"], s["n"], s["w"], s["block"], s["at"], s["slots"], s["codes"], s["w"],
                            s["scales"], s["scales"].shape[1])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    out = s["out"]
    if s["op"] == "read":
        csa.csa_dequantize_f8(kind[out.dtype], s["codes"], s["w"], s["scales"], s["scales"].shape[1], s["slots"], s["w"], s["block"],
                              s["at"], s["n"], out, s["w"])
    elif s["op"] == "gemm":
        M, N, K = s["M"], s["N"], s["K"]
        if "ws" not in s:
            s["ws"] = torch.empty(csa.csa_gemm_f8_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
        csa.csa_gemm_f8(kind[out.dtype], s["a"], K, s["sa"], s["sa"].shape[1], s["b"], K, s["sb"], s["sb"].shape[1], M, N, K, out, N,
                        s["ws"])
    else:
        if "ws" not in s:
            s["dims"] = csa.Dims(d=4096, c=512, m=4, cI=128, nhI=64, nh=s["nh"], dc=1536, topk=s["k"], dtype=csa.CSA_BF16)
            s["ws"] = torch.empty(csa.csa_mqa_f8_workspace_bytes(s["dims"], s["rows"]), dtype=torch.uint8, device=DEV)
        if s["decode"]:
            csa.csa_decode_mqa_f8(s["dims"], s["q"], s["nh"] * 512, s["codes"], s["scales"], s["idx"], s["pos"], s["cap"], s["rows"],
                                  out, s["ws"])
        else:
            csa.csa_sparse_mqa_f8(s["dims"], s["q"], s["nh"] * 512, s["codes"], s["scales"], s["idx"], s["cu"], s["cb"],
                                  s["cu"].numel() - 1, s["rows"], s["codes"].shape[0], out, s["ws"])
    return out


# ------------------------------------------------------------------ the definitions, in 64 bits
def _value64(codes):
    """Sign, four exponent bits and three fraction bits, bias 7, subnormals of 2^-9."""
    c = codes.long()
    ex, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(ex == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((ex - 7).double()))
    return torch.where(c >= 128, -v, v)


def _entries64(codes, byte, block):
    scale = torch.exp2(byte.double() - 127)
    col = torch.arange(codes.shape[-1], device=codes.device) // block
    return _value64(codes) * scale[..., col]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        x, n, w = s["x"].double(), case["n"], case["w"]
        block = case["block"] or w
        codes, byte = _value64(s["codes"]), s["scales"].long()
        at = torch.arange(n, device=DEV) if s["at"] is None else s["at"].long()
        for j in range(0, w, block):
            part = x[:, j: j + block]
            top = part.abs().amax(1)
            e = torch.ceil(torch.log2(top / 448))                    # the smallest e with top <= 448 * 2^e:
            e = torch.where(448 * torch.exp2(e - 1) >= top, e - 1, e)   # log2 may be a hair off at a border
            e = torch.where(448 * torch.exp2(e) < top, e + 1, e)
            e = torch.where(top > 0, e, -127.0).clamp(-127, 127)
            y = part / torch.exp2(e)[:, None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            codes[at, j: j + block] = torch.round(y / step) * step
            byte[at, j // block] = e.long() + 127
        return codes, byte.to(torch.uint8)
    if case["op"] == "read":
        v = _entries64(s["codes"], s["scales"], case["block"] or case["w"])
        return torch.where((s["at"] >= 0)[:, None], v[s["at"].long().clamp(min=0)], 0.0)
    if work(case)["flops"] > 3e11:     # over about 20 s in 64 bits
        return None
    if case["op"] == "gemm":
        a = _entries64(s["a"], s["sa"], 128)
        wide = s["sb"].long()[torch.arange(case["N"], device=DEV) // 128]
        return torch.matmul(a, _entries64(s["b"], wide, 128).t())
    rows, nh = case["rows"], case["nh"]
    out = torch.empty(rows, nh * 512, dtype=torch.float64, device=DEV)
    q = s["q"].view(rows, nh, 512)
    for r in range(0, rows, 64):
        idx = s["idx"][r: r + 64].long()
        at = s["base"][r: r + 64, None] + idx.clamp(min=0)
        e = _entries64(s["codes"][at], s["scales"][at][..., None], 512)
        t = torch.einsum("rhc,rsc->rhs", q[r: r + 64].double(), e) / math.sqrt(512)
        t = torch.where((idx >= 0)[:, None], t, -math.inf)
        none = (idx < 0).all(1)
        t = torch.where(none[:, None, None], 0.0, t)
        o = torch.einsum("rhs,rsc->rhc", torch.softmax(t, -1), e)
        out[r: r + 64] = torch.where(none[:, None, None], 0.0, o).reshape(-1, nh * 512)
    return out
