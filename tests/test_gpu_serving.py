"""GPU parity of the serving operators against their plain 64-bit forms (tests/serving_helpers.py):
prompt attention, the 4-bit cache's append, read, attention and eviction, and a run of them together.

Tolerances.  u = 2**-24 (float32, half a step) and 2**-8 (bfloat16).  A score is a product of d_h terms
summed in float32, then scaled: off by at most (d_h + 4) steps of sum |q_i k_i| * sm_scale; tensor cores
may truncate, so a step counts as 2 u.  A probability is then off by a factor of at most
e = 2 * (score error) + (n + 16) * 2 u (numerator and denominator see the scores, the sums have n terms).
So a weight is off by e * weight, and an output by (e + p) * sum_j P_ij |v_j|, p the rounding of P before
the product with V (2**-8 where it is bfloat16), then its own rounding.  float32 sums of the outputs'
n terms are inside e.
"""
import numpy as np
import pytest
import torch

import serving_helpers as R
from gpu_helpers import BF, lib

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
F32 = torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ws(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


def offsets(lens, first=0):
    return [first] + (first + np.cumsum(lens)).astype(int).tolist() if len(lens) else [first]


def score_step(q, k, n):
    """The factor e of the module's comment, from the largest sum |q_i k_i| of a (query, key) pair."""
    d = q.shape[-1]
    reach = np.sqrt((q ** 2).sum(-1).max(initial=0) * (k ** 2).sum(-1).max(initial=0)) / np.sqrt(d)   # Cauchy-Schwarz
    return 2 * (d + 4) * 2 * U32 * reach + (n + 16) * 2 * U32


def check_out(got, ref, spread, e, dtype, p_round, what=""):
    tol = (e + p_round) * spread
    tol = tol + (UBF if dtype == BF else U32) * (np.abs(ref) + tol) + 1e-37
    bad = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and bad.max(initial=-1) <= 0, f"{what}: off by {np.abs(got - ref).max()} (past its bound by {bad.max()})"


def check_weight(got, old, add, e, what=""):
    """weight = old + add in one float32 addition, add off by a factor of at most e."""
    bad = np.abs(got - (old + add)) - (e * add + 2 * U32 * (old + add) + 1e-37)
    assert bad.max(initial=-1) <= 0, f"{what}: weights past their bound by {bad.max()}"


# ---- prompt attention -------------------------------------------------------------------------------
class Prompt:
    def __init__(self, S, dtype, d, H, Hk, lens, kv, seed=0, front=0, back=0, wide=0, cap=None, kernel=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.S, self.dtype, self.cu_q, self.cu_kv = S, dtype, offsets(lens, front), offsets(kv, front)
        rq, rk = self.cu_q[-1] + back, self.cu_kv[-1] + back
        rnd = lambda r, h: torch.randn((r, h * d + wide), generator=g, device="cuda").to(dtype)
        self.qb, self.kb, self.vb = rnd(rq, H), rnd(rk, Hk), rnd(rk, Hk)
        self.kb[..., ::16] *= 3
        view = lambda t, h: t[:, :h * d].unflatten(1, (h, d))
        self.q, self.k, self.v = view(self.qb, H), view(self.kb, Hk), view(self.vb, Hk)
        self.o = view(torch.full((rq, H * d + wide), 7.0, dtype=dtype, device="cuda"), H)
        self.n_w = cap or max(max(kv, default=1), 1) + 3
        self.w0 = torch.rand((len(lens), Hk, self.n_w), generator=g, device="cuda")
        self.w, self.status = self.w0.clone(), i32([0])
        self.args = S.make_prompt_args(self.q, self.k, self.v, self.o, i32(self.cu_q), i32(self.cu_kv), weight=self.w,
                                       dev_status=self.status, kernel=kernel)
        self.nb = S.prompt_workspace_size(self.args)
        self.ws = ws(self.nb)

    def run(self):
        self.S.prompt_attention(self.args, self.ws, self.nb)
        torch.cuda.synchronize()
        return self

    def check(self, p_round, status=0, what=""):
        q, k, v = host(self.q), host(self.k), host(self.v)
        clean = lambda x: np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)
        n = max((b - a for a, b in zip(self.cu_kv, self.cu_kv[1:])), default=0)
        inside = slice(self.cu_kv[0], self.cu_kv[-1])
        e = score_step(clean(q[self.cu_q[0]:self.cu_q[-1]]), clean(k[inside]), n)
        ref, w = R.prompt_attention(q, k, v, self.cu_q, self.cu_kv, self.n_w)
        spread, _ = R.prompt_attention(q, k, np.abs(v), self.cu_q, self.cu_kv, self.n_w)
        own = slice(self.cu_q[0], self.cu_q[-1])
        check_out(host(self.o)[own], ref[own], spread[own], e, self.dtype, p_round, what)
        rest = np.r_[host(self.o)[:self.cu_q[0]], host(self.o)[self.cu_q[-1]:]]
        assert (rest == 7.0).all(), "rows outside every sequence were written"
        check_weight(host(self.w), host(self.w0), w, e, what)
        assert int(self.status.item()) == status
        return self


CASES = [  # dtype, d, H, Hk, query rows, key rows
    (BF, 64, 4, 4, [37], [37]), (BF, 128, 8, 2, [1], [1]), (BF, 64, 6, 2, [128, 256, 129, 1, 0, 300], [128, 256, 129, 1, 0, 300]),
    (BF, 128, 4, 1, [257, 33], [257, 33]), (BF, 128, 3, 3, [5, 400, 64], [261, 912, 64]), (BF, 64, 8, 1, [1, 130], [515, 131]),
    (BF, 64, 2, 2, [70, 3, 9], [20, 0, 9]), (BF, 128, 2, 1, [300, 140], [45, 139]), (BF, 128, 8, 8, [700], [700]),
    (F32, 64, 2, 1, [200, 65, 500], [200, 130, 577]), (F32, 128, 4, 2, [129, 40, 300], [321, 40, 700]),
    (F32, 64, 4, 4, [128, 1, 61], [128, 1, 61]), (F32, 128, 6, 2, [33, 65], [100, 65]), (F32, 64, 2, 1, [40, 5], [7, 0]),
]


@pytest.mark.parametrize("dtype,d,H,Hk,lens,kv", CASES)
def test_prompt(cuda, dtype, d, H, Hk, lens, kv):
    p = Prompt(lib(), dtype, d, H, Hk, lens, kv, seed=sum(lens) + d).run()
    p.check(UBF if dtype == BF else 0.0)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
def test_prompt_strides_and_rows_outside(cuda, dtype, d):
    """Row strides wider than the heads, rows before, between and behind the sequences' blocks."""
    Prompt(lib(), dtype, d, 4, 2, [60, 190], [60, 200], seed=5, front=3, back=11, wide=16).run().check(UBF if dtype == BF else 0.0)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_cuda_core_kernel_agrees(cuda, d):
    Prompt(lib(), BF, d, 4, 2, [150, 31], [150, 90], seed=6, kernel=1).run().check(0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_nonfinite_rows_of_others(cuda, dtype):
    """NaN and infinities in the rows around a sequence change nothing in it."""
    S = lib()
    p = Prompt(S, dtype, 128, 2, 1, [50, 70, 40], [50, 130, 40], seed=8, front=4, back=9)
    for t, cu in ((p.qb, p.cu_q), (p.kb, p.cu_kv), (p.vb, p.cu_kv)):
        t[:cu[0]] = float("nan")
        t[cu[3]:] = float("inf")
        t[cu[1]:cu[2]] = float("nan")
    p.run()
    ref, w = R.prompt_attention(host(p.q), host(p.k), host(p.v), p.cu_q, p.cu_kv, p.n_w)
    spread, _ = R.prompt_attention(host(p.q), host(p.k), np.abs(host(p.v)), p.cu_q, p.cu_kv, p.n_w)
    for b in (0, 2):
        rows, keys = slice(p.cu_q[b], p.cu_q[b + 1]), slice(p.cu_kv[b], p.cu_kv[b + 1])
        e = score_step(host(p.q)[rows], host(p.k)[keys], 50)
        check_out(host(p.o)[rows], ref[rows], spread[rows], e, dtype, UBF if dtype == BF else 0.0)
        check_weight(host(p.w)[b], host(p.w0)[b], w[b], e)


def test_prompt_large_scores(cuda):
    """Scores in the hundreds: one key takes nearly all of each row, and the sums stay finite."""
    S = lib()
    for dtype in (BF, F32):
        p = Prompt(S, dtype, 64, 2, 2, [200], [200], seed=9)
        p.qb *= 30
        p.run().check(UBF if dtype == BF else 0.0)


def test_prompt_bad_offsets_and_short_weight(cuda):
    S = lib()
    for dtype in (BF, F32):
        p = Prompt(S, dtype, 64, 2, 2, [20, 30], [20, 30], seed=10)
        good = p.cu_q
        for bad in ([0, 20, 51], [0, -1, 50], [30, 20, 50]):
            p.args.cu_q = (t := i32(bad)).data_ptr()
            p.status.zero_()
            p.run()
            assert int(p.status.item()) == S.E_INDEX, bad
            assert torch.isfinite(p.o.float()).all()
        del t
        p = Prompt(S, dtype, 64, 2, 2, [20, 30], [20, 30], seed=10, cap=25)
        p.run().check(UBF if dtype == BF else 0.0, status=S.E_INDEX)
        assert good == p.cu_q


def test_prompt_replayed_on_another_stream(cuda):
    """A captured call replayed on another stream gives the eager call's bits, every time."""
    S = lib()
    p = Prompt(S, BF, 128, 4, 2, [90, 300], [90, 310], seed=11).run()
    o, w = p.o.clone(), p.w.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        S.prompt_attention(p.args, p.ws, p.nb)
    for _ in range(2):
        p.o.fill_(0)
        p.w.copy_(p.w0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.o, o) and torch.equal(p.w, w)


# ---- the 4-bit cache -----------------------------------------------------------------------------------
class Cache:
    """A cache with random contents, and what its first n rows hold as host arrays."""

    def __init__(self, S, B, H, d, cap, seed=0):
        r = np.random.default_rng(seed)
        self.S, self.B, self.H, self.d, self.cap = S, B, H, d, cap
        code = lambda: r.integers(-7, 8, (B, H, cap, d))
        scale = lambda: R.to_bf16(np.exp(r.normal(0, 0.5, (B, H, cap, d // 32))))
        dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()
        self.t = {"k_codes": dev(R.pack4(code(), 8), torch.uint8), "k_scale": dev(scale(), BF),
                  "v_codes": dev(R.pack4(code(), 4), torch.uint8), "v_scale": dev(scale(), BF),
                  "weight": dev(r.exponential(1, (B, H, cap)), F32), "pos": dev(np.tile(np.arange(cap), (B, H, 1)), torch.int32)}
        self.c = S.make_kv4_cache(**self.t)

    def host(self):
        return {k: (v.float() if v.dtype == BF else v).cpu().numpy() for k, v in self.t.items()}

    def values(self):
        h = self.host()
        return R.values4(h["k_codes"], h["k_scale"], 8), R.values4(h["v_codes"], h["v_scale"], 4)


@pytest.mark.parametrize("dtype,B,H,d,lens,old", [
    (BF, 1, 1, 64, [5], [0]), (BF, 3, 4, 128, [33, 0, 70], [7, 100, 2]), (F32, 2, 3, 64, [17, 40], [0, 9]),
    (F32, 2, 2, 128, [1, 1], [3, 0]), (BF, 4, 12, 64, None, [5, 0, 99, 39]), (F32, 2, 5, 128, None, [0, 1])])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(cuda, dtype, B, H, d, lens, old, in_place):
    """Codes, scales, weights, positions and counts, exact; every other row of the cache stays."""
    S = lib()
    cap = 110
    c = Cache(S, B, H, d, cap, seed=d + B)
    before = c.host()
    cu = [0, *range(1, B + 1)] if lens is None else offsets(lens)
    rows = cu[-1] + (0 if lens is None else 4)          # rows behind the last sequence are ignored
    g = torch.Generator(device="cuda").manual_seed(3)
    x = [torch.randn((rows, 2 * H * d), generator=g, device="cuda").to(dtype) for _ in range(2)]
    x[0][0, :32] = 0                                     # a group of zeros
    if rows > 1:
        x[0][1, :8] = torch.tensor([7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, 6.5], device="cuda").to(dtype)
        x[0][1, 8:32] = 0                                # scale 1: halves round to even
    ln, seen = i32(old), i32([o + 1000 for o in old])
    lo, so = (ln, seen) if in_place else (torch.zeros_like(ln), torch.zeros_like(seen))
    status = i32([0])
    S.kv4_append(c.c, x[0], x[1], 2 * H * d, rows, ln, lo, seen, so, cu=None if lens is None else i32(cu), dev_status=status)
    torch.cuda.synchronize()
    want = before
    for b in range(B):
        n = cu[b + 1] - cu[b]
        at = slice(old[b], old[b] + n)
        for t, name, run in ((0, "k", 8), (1, "v", 4)):
            xv = x[t][cu[b]:cu[b + 1], :H * d].float().cpu().numpy().reshape(n, H, d)
            code, s = R.quantize4(xv)
            want[name + "_codes"][b, :, at] = R.pack4(code, run).transpose(1, 0, 2)
            want[name + "_scale"][b, :, at] = s.transpose(1, 0, 2)
        want["weight"][b, :, at] = 0
        want["pos"][b, :, at] = old[b] + 1000 + np.arange(n)
    got = c.host()
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    n = np.diff(cu)
    assert lo.tolist() == (np.array(old) + n).tolist() and so.tolist() == (np.array(old) + 1000 + n).tolist()
    assert int(status.item()) == 0


def test_append_past_capacity_and_nonfinite(cuda):
    S = lib()
    for cu, ln in (([0, 6, 12], [6, 2]), (None, [10, 4])):
        c = Cache(S, 2, 2, 64, 10, seed=1)
        rows = 12 if cu else 2
        x = torch.randn((rows, 2, 64), device="cuda")
        n, seen, status = i32(ln), i32([50, 60]), i32([0])
        S.kv4_append(c.c, x, x, 128, rows, n, n, seen, seen, cu=i32(cu) if cu else None, dev_status=status)
        assert int(status.item()) == S.E_INDEX
        assert n.tolist() == ([10, 8] if cu else [10, 5]) and seen.tolist() == ([54, 66] if cu else [50, 61])
    c = Cache(S, 1, 1, 64, 4, seed=2)
    x = torch.randn((1, 1, 64), device="cuda")
    x[0, 0, 3], x[0, 0, 40], x[0, 0, 41] = float("nan"), float("inf"), float("-inf")
    n, status = i32([0]), i32([0])
    S.kv4_append(c.c, x, x, 64, 1, n, n, n.clone(), n.clone(), dev_status=status)
    code, s = R.quantize4(x.cpu().numpy())
    np.testing.assert_array_equal(c.host()["k_codes"][0, 0, 0], R.pack4(code[0, 0], 8))
    assert int(status.item()) == S.E_NONFINITE


def test_append_range(cuda):
    """The whole range of float32: subnormal rows, the largest values, signed zeros."""
    S = lib()
    r = np.random.default_rng(4)
    x = (r.standard_normal((40, 1, 64)) * np.exp2(np.linspace(-149, 126, 40))[:, None, None]).astype(np.float32)
    x[0], x[1, 0, :32] = -0.0, np.float32(1e-45)
    c, n, status = Cache(S, 1, 1, 64, 40, seed=3), i32([0]), i32([0])
    t = torch.from_numpy(x).cuda()
    S.kv4_append(c.c, t, t, 64, 40, n, n, n.clone(), n.clone(), cu=i32([0, 40]), dev_status=status)
    code, s = R.quantize4(x)
    got = c.host()
    np.testing.assert_array_equal(got["k_scale"][0, 0], s[:, 0])
    np.testing.assert_array_equal(got["k_codes"][0, 0], R.pack4(code[:, 0], 8))
    np.testing.assert_array_equal(got["v_codes"][0, 0], R.pack4(code[:, 0], 4))
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
def test_read(cuda, dtype, d):
    S = lib()
    c = Cache(S, 3, 2, d, 50, seed=d)
    k, v = c.values()
    cu, row0 = [2, 9, 9, 30], [40, 0, 10]
    out = [torch.full((33, 2 * d + 8), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    status = i32([0])
    S.kv4_read(c.c, i32(cu), 33, out[0], out[1], 2 * d + 8, row0=i32(row0), dev_status=status)
    torch.cuda.synchronize()
    for o, x in zip(out, (k, v)):
        want = np.full((33, 2 * d + 8), 7.0)
        for b in range(3):
            n = cu[b + 1] - cu[b]
            rows = x[b][:, row0[b]:row0[b] + n].transpose(1, 0, 2).reshape(n, 2 * d)
            want[cu[b]:cu[b + 1], :2 * d] = R.to_bf16(rows) if dtype == BF else rows
        np.testing.assert_array_equal(host(o), want)
    assert int(status.item()) == 0
    S.kv4_read(c.c, i32(cu), 33, out[0], None, 2 * d + 8, row0=i32([45, 0, 0]), dev_status=status)
    assert int(status.item()) == S.E_INDEX and (host(out[0])[7:9, :2 * d] == 0).all()


def run_attention(S, c, q, n, n_max=None, update=True, o=None, w=None):
    o = torch.empty_like(q) if o is None else o
    status = i32([0])
    ln = i32(n)
    a = S.make_kv4_attn_args(c.c, q, o, ln, n_max or c.cap, update, dev_status=status)
    nb = S.kv4_attention_workspace_size(a)
    S.kv4_attention(a, ws(nb) if w is None else w, nb)
    torch.cuda.synchronize()
    return o, int(status.item())


@pytest.mark.parametrize("dtype,B,H,Hk,d,cap,n", [
    (BF, 1, 1, 1, 64, 1, [1]), (BF, 3, 4, 4, 64, 70, [70, 0, 17]), (BF, 2, 8, 2, 128, 333, [333, 16]),
    (BF, 2, 16, 1, 128, 129, [129, 15]), (BF, 1, 24, 2, 64, 1500, [1499]), (BF, 1, 40, 1, 128, 200, [200]),
    (F32, 2, 3, 3, 64, 65, [64, 65]), (F32, 2, 12, 2, 128, 300, [33, 300]), (F32, 1, 34, 2, 64, 100, [100]),
    (BF, 1, 2, 2, 128, 9000, [8999]), (BF, 5, 6, 2, 64, 260, [256, 255, 257, 1, 2])])
def test_attention(cuda, dtype, B, H, Hk, d, cap, n):
    S = lib()
    c = Cache(S, B, Hk, d, cap, seed=cap + H)
    g = torch.Generator(device="cuda").manual_seed(cap)
    qb = torch.randn((B, H * d + 24), generator=g, device="cuda").to(dtype)
    q = qb[:, :H * d].unflatten(1, (H, d))
    w0 = c.t["weight"].clone()
    o, status = run_attention(S, c, q, n)
    assert status == 0
    k, v = c.values()
    got_w = host(c.t["weight"])
    for b in range(B):
        ref, w = R.kv4_attention(host(q)[b], k[b], v[b], n[b])
        spread, _ = R.kv4_attention(host(q)[b], k[b], np.abs(v[b]), n[b])
        e = score_step(host(q)[b], k[b], n[b])
        check_out(host(o)[b], ref, spread, e, dtype, UBF if dtype == BF else 2 * U32, f"sequence {b}")
        check_weight(got_w[b], host(w0)[b], w, e)
        assert (got_w[b][:, n[b]:] == host(w0)[b][:, n[b]:]).all()


def test_attention_lengths_out_of_range_and_no_update(cuda):
    S = lib()
    c = Cache(S, 3, 2, 64, 90, seed=7)
    q = torch.randn((3, 4, 64), device="cuda")
    w0 = c.t["weight"].clone()
    a, s = run_attention(S, c, q, [95, -3, 40], n_max=80, update=False)
    b, t = run_attention(S, c, q, [80, 0, 40], n_max=80, update=False)
    assert s == S.E_INDEX and t == 0 and torch.equal(a, b) and (a[1] == 0).all()
    assert torch.equal(w0, c.t["weight"])


def test_attention_large_scores_and_scales(cuda):
    """Scales over many binades and scores in the thousands: finite, and within the bounds."""
    S = lib()
    for dtype in (BF, F32):
        c = Cache(S, 1, 1, 128, 77, seed=8)
        c.t["k_scale"][:, :, ::3] *= 64
        c.t["v_scale"][:, :, 1::2] *= 2.0 ** -40
        c.t["v_scale"][:, :, ::5] *= 2.0 ** 30
        q = (4 * torch.randn((1, 3, 128), device="cuda")).to(dtype)
        o, _ = run_attention(S, c, q, [77], update=False)
        k, v = c.values()
        ref, _ = R.kv4_attention(host(q)[0], k[0], v[0], 77)
        spread, _ = R.kv4_attention(host(q)[0], k[0], np.abs(v[0]), 77)
        check_out(host(o)[0], ref, spread, score_step(host(q)[0], k[0], 77), dtype, UBF if dtype == BF else 2 * U32)


def test_attention_bits_repeat_and_replay(cuda):
    """Reruns, another stream and a replayed capture give the same bits; two captured calls of their own
    workspaces may run at once."""
    S = lib()
    c = Cache(S, 2, 4, 128, 700, seed=9)
    q = torch.randn((2, 16, 128), device="cuda").to(BF)
    w0 = c.t["weight"].clone()
    o, _ = run_attention(S, c, q, [700, 333])
    w = c.t["weight"].clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    o2, ln = torch.empty_like(o), i32([700, 333])
    a = S.make_kv4_attn_args(c.c, q, o2, ln, 700)
    nb = S.kv4_attention_workspace_size(a)
    w1 = ws(nb)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        S.kv4_attention(a, w1, nb)
    for _ in range(2):
        c.t["weight"].copy_(w0)
        w1.fill_(255)                                    # nothing in the workspace is read before it is written
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(w, c.t["weight"])


@pytest.mark.parametrize("d,n,keep,recent,in_place", [
    (64, [90, 40, 41], 40, 0, True), (64, [90, 40, 41], 40, 7, False), (128, [2500, 1, 0], 700, 100, True),
    (128, [2500, 30, 1300], 1200, 1200, False), (64, [1025, 1024, 3], 1, 1, True), (64, [300, 299, 298], 299, 0, False),
    (64, [50, 60, 70], 90, 5, False)])
def test_evict(cuda, d, n, keep, recent, in_place):
    """Which rows stay and where they end up, exact: ties, infinities, equal weights, recent rows."""
    S = lib()
    H, cap = 3, max(n) + 2
    c = Cache(S, 3, H, d, cap, seed=keep)
    r = np.random.default_rng(keep)
    w = np.round(r.exponential(3, (3, H, cap)) * 2).astype(np.float32) / 2       # many ties
    w[:, 0] *= np.where(r.random((3, cap)) < 0.5, -1, 1)                         # -0.0 and negative weights too
    w[0, 1, :5], w[1, 1] = [np.inf, -np.inf, 0, np.inf, -0.0], 1.0               # infinities, all equal
    c.t["weight"].copy_(torch.from_numpy(w))
    c.t["pos"].copy_(torch.from_numpy(np.stack([np.stack([r.permutation(cap) for _ in range(H)]) for _ in range(3)]).astype(np.int32)))
    before = c.host()
    dst = c if in_place else Cache(S, 3, H, d, keep + 1, seed=1)
    other = dst.host()
    ln, seen, status = i32(n), i32([cap] * 3), i32([0])
    out = ln if in_place else torch.zeros_like(ln)
    nb = S.kv4_evict_workspace_size(c.c, cap, keep)
    S.kv4_evict(c.c, dst.c, ln, out, seen, cap, keep, recent, ws(nb), nb, dev_status=status)
    torch.cuda.synchronize()
    got = dst.host()
    for b in range(3):
        for h in range(H):
            src = R.evict_sources(before["weight"][b, h], before["pos"][b, h], n[b], cap, keep, recent)
            for key in got:
                np.testing.assert_array_equal(got[key][b, h, :len(src)], before[key][b, h, src], err_msg=f"{key} {b} {h}")
                if not in_place:                          # rows behind the kept ones stay
                    np.testing.assert_array_equal(got[key][b, h, len(src):], other[key][b, h, len(src):])
    assert out.tolist() == [min(x, keep) for x in n] and int(status.item()) == 0
    if not in_place:
        for key, x in c.host().items():
            np.testing.assert_array_equal(x, before[key])


def test_evict_nan_and_lengths(cuda):
    S = lib()
    c = Cache(S, 2, 1, 64, 40, seed=5)
    c.t["weight"][0, 0, 3] = float("nan")
    before = c.host()
    ln, status = i32([50, 40]), i32([0])
    nb = S.kv4_evict_workspace_size(c.c, 40, 10)
    S.kv4_evict(c.c, c.c, ln, ln, None, 40, 10, 0, ws(nb), nb, dev_status=status)
    assert int(status.item()) in (S.E_INDEX, S.E_NONFINITE) and ln.tolist() == [10, 10]
    for b in range(2):
        src = R.evict_sources(before["weight"][b, 0], None, 40, 0, 10, 0)
        np.testing.assert_array_equal(c.host()["k_codes"][b, 0, :10], before["k_codes"][b, 0, src])


def test_rows_past_4_gib(cuda):
    """Planes of more than 2**32 bytes: append, read and attention at their far end."""
    S = lib()
    cap = (1 << 26) + 37
    new = lambda tail, dt: torch.zeros((1, 1, cap) + tail, dtype=dt, device="cuda")
    t = [new((64,), torch.uint8), new((4,), BF), new((64,), torch.uint8), new((4,), BF)]
    c = S.make_kv4_cache(*t)
    x = torch.randn((5, 1, 128), device="cuda")
    y = torch.randn((5, 1, 128), device="cuda")
    n, status = i32([cap - 5]), i32([0])
    S.kv4_append(c, x, y, 128, 5, n, n, cu=i32([0, 5]), dev_status=status)
    out = torch.empty_like(x), torch.empty_like(x)
    S.kv4_read(c, i32([0, 5]), 5, out[0], out[1], 128, row0=i32([cap - 5]), dev_status=status)
    for o, src in zip(out, (x, y)):
        code, s = R.quantize4(src.cpu().numpy())
        np.testing.assert_array_equal(host(o)[:, 0], (code * np.repeat(s, 32, -1))[:, 0])
    # every other row is 0 in K and V (code 0x00 is -8 with scale 0): the far rows take what e^s gives them
    q = (40 * out[0][2, 0] / out[0][2, 0].norm())[None, None].contiguous()
    o = torch.empty_like(q)
    a = S.make_kv4_attn_args(c, q, o, n, cap, update_weight=False, dev_status=status)
    nb = S.kv4_attention_workspace_size(a)
    S.kv4_attention(a, ws(nb), nb)
    torch.cuda.synchronize()
    sc = np.r_[host(out[0])[:, 0] @ host(q)[0, 0] / np.sqrt(128), 0.0]
    p = np.exp(sc - sc.max()) * np.r_[np.ones(5), cap - 5]
    ref = (p[:5] / p.sum()) @ host(out[1])[:, 0]
    spread = (p[:5] / p.sum()) @ np.abs(host(out[1])[:, 0])
    check_out(host(o)[0, 0], ref, spread, score_step(host(q)[0], host(out[0])[:, 0], 5), F32, 2 * U32)
    assert int(status.item()) == 0 and n.tolist() == [cap]


# ---- together ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,H,Hk", [(BF, 64, 4, 4), (BF, 128, 8, 2), (F32, 64, 6, 2)])
def test_generation_with_eviction(cuda, dtype, d, H, Hk):
    """Prompts, an eviction, generated tokens (a captured step, replayed), an eviction, and a second turn
    over what is left; every output against the plain forms on the device's own cache."""
    from cascade_token_head_b200.kv4 import KV4State
    S = lib()
    B, lens, keep, recent = 2, [75, 130], 60, 10
    st = KV4State(B, H, Hk, d, 256)
    g = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda r, h: torch.randn((r, h, d), generator=g, device="cuda").to(dtype)
    cu = offsets(lens)
    q, k, v = rnd(205, H), rnd(205, Hk), rnd(205, Hk)
    o = st.prompt(q, k, v, i32(cu))
    pr = UBF if dtype == BF else 2 * U32
    ref, w = R.prompt_attention(host(q), host(k), host(v), cu, cu, 256)
    spread, _ = R.prompt_attention(host(q), host(k), np.abs(host(v)), cu, cu, 256)
    e = score_step(host(q), host(k), 130)
    check_out(host(o), ref, spread, e, dtype, pr, "prompt")
    check_weight(host(st.weight), 0.0, w, e)
    assert st.len.tolist() == lens

    def cached():
        t = lambda x: (x.float() if x.dtype == BF else x).cpu().numpy()
        return R.values4(t(st.k_codes), t(st.k_scale), 8), R.values4(t(st.v_codes), t(st.v_scale), 4)

    def evict():
        w, p, n, seen = host(st.weight), st.pos.cpu().numpy(), st.len.tolist(), st.seen.tolist()
        old = cached()
        st.evict(keep, recent)
        for b in range(B):
            for h in range(Hk):
                src = R.evict_sources(w[b, h].astype(np.float32), p[b, h], n[b], seen[b], keep, recent)
                assert st.pos[b, h, :len(src)].tolist() == p[b, h, src].tolist()
                for a, x in zip(old, cached()):
                    np.testing.assert_array_equal(x[b, h, :len(src)], a[b, h, src])
        assert st.len.tolist() == [min(x, keep) for x in n]
    evict()

    x = [rnd(B, H), rnd(B, Hk), rnd(B, Hk)]
    out = torch.empty_like(x[0])
    st.step(*x, o=out)                                    # once eagerly, then captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.step(*x, o=out)
    assert st.len.tolist() == [keep + 1] * B
    for _ in range(12):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        w0 = host(st.weight)
        graph.replay()
        torch.cuda.synchronize()
        kk, vv = cached()
        for b in range(B):
            n = int(st.len[b])
            ref, w = R.kv4_attention(host(x[0])[b], kk[b], vv[b], n)
            spread, _ = R.kv4_attention(host(x[0])[b], kk[b], np.abs(vv[b]), n)
            e = score_step(host(x[0])[b], kk[b][:, :n], n)
            check_out(host(out)[b], ref, spread, e, dtype, pr, "step")
            w0[b, :, n - 1] = 0
            check_weight(host(st.weight)[b, :, :n], w0[b, :, :n], w[:, :n], e)
    evict()

    n_old, new = st.len.tolist(), [9, 1]
    cu2, cu_kv = offsets(new), offsets([a + b for a, b in zip(n_old, new)])
    q, k, v = rnd(10, H), rnd(10, Hk), rnd(10, Hk)
    o = st.resume(q, k, v, i32(cu2), i32(cu_kv), cu_kv[-1])
    kk, vv = cached()
    rows = lambda x: np.concatenate([x[b, :, :n_old[b] + new[b]].transpose(1, 0, 2) for b in range(B)])
    kk, vv = (R.to_bf16(rows(x)) if dtype == BF else rows(x) for x in (kk, vv))
    ref, _ = R.prompt_attention(host(q), kk, vv, cu2, cu_kv, 1)
    spread, _ = R.prompt_attention(host(q), kk, np.abs(vv), cu2, cu_kv, 1)
    check_out(host(o), ref, spread, score_step(host(q), kk, 70), dtype, pr, "second turn")
    assert st.seen.tolist() == [lens[b] + 13 + new[b] for b in range(B)] and int(st.status.item()) == 0


@pytest.mark.parametrize("d,H", [(64, 2), (128, 4)])
def test_prompt_forced_timeout_reports_status_and_context_survives(cuda, d, H):
    """One poll per wait: the kernels give up, say so, and the next call is whole."""
    S = lib()
    p = Prompt(S, BF, d, H, 2, [600, 90], [700, 90], seed=21)
    try:
        S.set_wait_limit(1)
        p.run()
        assert int(p.status.item()) == S.E_TIMEOUT
    finally:
        S.set_wait_limit(0)
    p.status.zero_()
    p.w.copy_(p.w0)
    p.run().check(UBF)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 128)])
def test_attention_scores_in_the_workspace(cuda, dtype, d):
    """Sixteen heads over 20,000 keys: the scores do not fit the SMs' shared memory."""
    S = lib()
    n = [20000]
    c = Cache(S, 1, 1, d, n[0], seed=31)
    q = torch.randn((1, 16, d), device="cuda").to(dtype)
    a = S.make_kv4_attn_args(c.c, q, torch.empty_like(q), i32(n), n[0])
    assert S.kv4_attention_workspace_size(a) >= 16 * n[0] * 4
    w0 = c.t["weight"].clone()
    o, status = run_attention(S, c, q, n)
    assert status == 0
    k, v = c.values()
    ref, w = R.kv4_attention(host(q)[0], k[0], v[0], n[0])
    spread, _ = R.kv4_attention(host(q)[0], k[0], np.abs(v[0]), n[0])
    e = score_step(host(q)[0], k[0], n[0])
    check_out(host(o)[0], ref, spread, e, dtype, UBF if dtype == BF else 2 * U32)
    check_weight(host(c.t["weight"])[0], host(w0)[0], w, e)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_more_rows_than_shared_memory_holds(cuda, in_place):
    """60,000 rows: the selection reads the weights themselves; many rows of one weight."""
    S = lib()
    n, keep, recent, d = [60000, 59999], 30001, 77, 64
    cap = 60000
    c = Cache(S, 2, 1, d, cap, seed=5)
    r = np.random.default_rng(1)
    w = np.zeros((2, 1, cap), np.float32)
    w[0] = r.exponential(1, (1, cap))
    w[1, 0, ::3] = 1.0
    pos = np.tile(np.arange(cap, dtype=np.int32), (2, 1, 1))
    c.t["weight"].copy_(torch.from_numpy(w))
    c.t["pos"].copy_(torch.from_numpy(pos))
    before = c.host()
    dst = c if in_place else Cache(S, 2, 1, d, keep, seed=1)
    ln, status = i32(n), i32([0])
    lo = ln if in_place else torch.zeros_like(ln)
    nb = S.kv4_evict_workspace_size(c.c, cap, keep)
    S.kv4_evict(c.c, dst.c, ln, lo, i32(n), cap, keep, recent, ws(nb), nb, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lo.tolist() == [keep, keep]
    got = dst.host()
    for b in range(2):
        src = R.evict_sources(w[b, 0], pos[b, 0], n[b], n[b], keep, recent)
        for k in before:
            np.testing.assert_array_equal(got[k][b, 0, :keep], before[k][b, 0, src], err_msg=k)


def test_calls_back_to_back_see_each_other(cuda):
    """A long run of dependent calls without a synchronisation: a kernel may start before the one ahead of it
    has ended, but sees all that it wrote.  Appends, evictions, attention and reads of one state."""
    S = lib()
    B, H, d, cap, rows = 3, 2, 64, 96, 8
    g = torch.Generator(device="cuda").manual_seed(77)
    k, v = (torch.randn((40, B * rows, H, d), generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((40, B, 4, d), generator=g, device="cuda").to(BF)

    def run(sync):
        c = Cache(S, B, H, d, cap, seed=3)
        c.t["weight"].zero_()
        ln, seen, status, cu = i32([0] * B), i32([0] * B), i32([0]), i32(offsets([rows] * B))
        nb = S.kv4_evict_workspace_size(c.c, cap, 50)
        w, out = ws(nb), []
        for i in range(40):
            S.kv4_append(c.c, k[i], v[i], H * d, B * rows, ln, ln, seen, seen, cu=cu, dev_status=status)
            o = torch.empty_like(q[i])
            a = S.make_kv4_attn_args(c.c, q[i], o, ln, cap, dev_status=status)
            na = S.kv4_attention_workspace_size(a)
            S.kv4_attention(a, ws(na), na)
            ko, vo = (torch.empty((B * 50, H, d), dtype=BF, device="cuda") for _ in range(2))
            S.kv4_evict(c.c, c.c, ln, ln, seen, cap, 50, 5, w, nb, status)
            S.kv4_read(c.c, i32(offsets([50] * B)), B * 50, ko, vo, H * d, dev_status=status)
            out += [o, ko, vo]
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return out + list(c.t.values()) + [ln, seen]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d,B,Hk,H,cap,n", [
    (BF, 64, 33, 16, 16, 300, [300, 0, 1] + [17 * i % 301 for i in range(30)]),     # many pairs, empty ones among them
    (BF, 128, 40, 8, 32, 260, [1] * 39 + [260]),                                    # nearly all in one sequence
    (F32, 64, 10, 32, 64, 280, [0] * 9 + [5]),                                      # fewer tiles than CTAs
    (BF, 128, 80, 4, 96, 150, [150 - i for i in range(80)]),                        # more heads than one pass takes
    (F32, 128, 75, 4, 4, 200, [200 - 2 * i for i in range(75)])])
def test_attention_dealt_over_the_gpu(cuda, dtype, d, B, Hk, H, cap, n):
    """More (sequence, head) pairs than one wave of CTAs: the keys are dealt in equal runs."""
    S = lib()
    c = Cache(S, B, Hk, d, cap, seed=B)
    q = torch.randn((B, H, d), device="cuda").to(dtype)
    w0 = c.t["weight"].clone()
    o, status = run_attention(S, c, q, n)
    assert status == 0
    k, v = c.values()
    got, got_w = host(o), host(c.t["weight"])
    for b in list(range(0, B, 7)) + [B - 1, 1]:
        ref, w = R.kv4_attention(host(q)[b], k[b], v[b], n[b])
        spread, _ = R.kv4_attention(host(q)[b], k[b], np.abs(v[b]), n[b])
        e = score_step(host(q)[b], k[b], n[b])
        check_out(got[b], ref, spread, e, dtype, UBF if dtype == BF else 2 * U32, f"sequence {b}")
        check_weight(got_w[b], host(w0)[b], w, e)
        assert (got_w[b][:, n[b]:] == host(w0)[b][:, n[b]:]).all()
    o2, _ = run_attention(S, c, q, n, update=False)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
@pytest.mark.parametrize("B", [32, 33, 70])
def test_prompt_many_sequences(cuda, dtype, d, B):
    """More sequences than a warp has lanes, some without rows, some going on over earlier rows."""
    r = np.random.default_rng(B + d)
    lens = r.integers(0, 160, B)
    lens[::7] = 0
    old = r.integers(0, 2, B) * r.integers(0, 150, B)
    Prompt(lib(), dtype, d, 2, 1, lens.tolist(), (lens + old).tolist(), seed=B).run().check(UBF if dtype == BF else 0.0)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_float32_on_cuda_cores(cuda, d):
    Prompt(lib(), F32, d, 4, 2, [150, 0, 65], [150, 20, 200], seed=16, kernel=1).run().check(0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_without_any_key(cuda, dtype):
    """No sequence has keys: outputs of zero, weights as they were."""
    Prompt(lib(), dtype, 64, 4, 2, [3, 70], [0, 0], seed=17).run().check(0.0)


@pytest.mark.parametrize("d", [64, 128])
def test_append_and_read_many_sequences(cuda, d):
    """Prompts of 70 sequences (more than a warp has lanes) into the cache and back: the quantized rows."""
    S, B, H = lib(), 70, 3
    r = np.random.default_rng(d)
    lens, old = r.integers(0, 40, B), r.integers(0, 9, B)
    lens[3::9] = 0
    c, cu = Cache(S, B, H, d, 50, seed=d), offsets(lens)
    x = [torch.randn((cu[-1], H, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(d)) for _ in range(2)]
    n, status = i32(old.tolist()), i32([0])
    S.kv4_append(c.c, x[0], x[1], H * d, cu[-1], n, n, n.clone(), n.clone(), cu=i32(cu), dev_status=status)
    out = [torch.empty_like(t) for t in x]
    S.kv4_read(c.c, i32(cu), cu[-1], out[0], out[1], H * d, row0=i32(old.tolist()), dev_status=status)
    assert n.tolist() == (old + lens).tolist() and int(status.item()) == 0
    for t, o, run in ((x[0], out[0], 8), (x[1], out[1], 4)):
        code, s = R.quantize4(t.cpu().numpy())
        np.testing.assert_array_equal(host(o), code.astype(np.float64) * np.repeat(s, 32, axis=-1).astype(np.float64))


def test_first_calls_are_captured(cuda):
    """A process whose first calls of the library are inside a graph capture; replays give the eager bits."""
    import os
    import subprocess
    import sys
    from pathlib import Path
    code = """
import torch
from cascade_token_head_b200 import kv4
def state():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn((90, h, 64), device="cuda", generator=g).to(torch.bfloat16) for h in (4, 2, 2)]
    t = [torch.randn((2, h, 64), device="cuda", generator=g).to(torch.bfloat16) for h in (4, 2, 2)]
    return kv4.KV4State(2, 4, 2, 64, 128), x, t, torch.empty_like(x[0]), torch.empty_like(t[0])
cu = torch.tensor([0, 50, 90], dtype=torch.int32, device="cuda")
def run(st, x, t, o, o1):
    st.prompt(*x, cu, o)
    st.evict(20, 4)
    st.step(*t, o1)
a, b = state(), state()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run(*a)
g.replay()
run(*b)
torch.cuda.synchronize()
for x, y in ((a[3], b[3]), (a[4], b[4]), (a[0].weight, b[0].weight), (a[0].k_codes, b[0].k_codes), (a[0].len, b[0].len)):
    assert torch.equal(x, y)
assert int(a[0].status) == int(b[0].status) == 0 and a[0].len.tolist() == [21, 21]
print("same bits")
"""
    root = str(Path(__file__).resolve().parent.parent)
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, PYTHONPATH=root), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift,wide", [(0, 4), (4, 0), (4, 4)])
def test_float32_rows_at_16_byte_addresses(cuda, d, shift, wide):
    """float32 rows whose addresses are multiples of 16 bytes, not of 32: append and read give the exact rows."""
    S, H, n = lib(), 3, 50
    ld = H * d + wide
    x = torch.randn((n * ld + shift,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(d + wide))
    rows = x[shift:].view(n, ld)
    c, ln, status = Cache(S, 2, H, d, 40, seed=d), i32([0, 3]), i32([0])
    S.kv4_append(c.c, rows, rows, ld, n, ln, ln, ln.clone(), ln.clone(), cu=i32([0, 21, 50]), dev_status=status)
    out = torch.full((n * ld + shift,), 7.0, device="cuda")
    got = out[shift:].view(n, ld)
    S.kv4_read(c.c, i32([0, 21, 50]), n, got, None, ld, row0=i32([0, 3]), dev_status=status)
    code, s = R.quantize4(rows[:, :H * d].unflatten(1, (H, d)).cpu().numpy())
    np.testing.assert_array_equal(host(got)[:, :H * d].reshape(n, H, d), code.astype(np.float64) * np.repeat(s, 32, axis=-1).astype(np.float64))
    assert (host(got)[:, H * d:] == 7).all() and (host(out)[:shift] == 7).all() and int(status.item()) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
def test_prompt_rows_at_16_byte_addresses(cuda, dtype, d):
    """Rows whose addresses are multiples of 16 bytes, not of 32."""
    Prompt(lib(), dtype, d, 3, 3, [60, 150], [60, 190], seed=18, front=1, back=2,
           wide=8 if dtype == BF else 4).run().check(UBF if dtype == BF else 0.0)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,top", [(25, 200), (50, 1100)])
def test_evict_many_heads(cuda, in_place, B, top):
    """More (sequence, head) pairs than two CTAs an SM hold."""
    S, H, d, keep, recent = lib(), 12, 64, 60, 9
    r = np.random.default_rng(B)
    n = r.integers(0, top, B)
    n[:3] = 0, keep, top
    cap = top + 1
    c = Cache(S, B, H, d, cap, seed=B)
    c.t["weight"].copy_(torch.round(c.t["weight"] * 8) / 8)      # ties
    before = c.host()
    dst = c if in_place else Cache(S, B, H, d, keep, seed=1)
    ln, status = i32(n.tolist()), i32([0])
    out = ln if in_place else torch.zeros_like(ln)
    nb = S.kv4_evict_workspace_size(c.c, cap, keep)
    S.kv4_evict(c.c, dst.c, ln, out, i32(n.tolist()), cap, keep, recent, ws(nb), nb, dev_status=status)
    torch.cuda.synchronize()
    got = dst.host()
    for b in range(B):
        for h in range(0, H, 5):
            src = R.evict_sources(before["weight"][b, h], before["pos"][b, h], int(n[b]), int(n[b]), keep, recent)
            for key in got:
                np.testing.assert_array_equal(got[key][b, h, :len(src)], before[key][b, h, src], err_msg=f"{key} {b} {h}")
    assert out.tolist() == np.minimum(n, keep).tolist() and int(status.item()) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("kernel", [0, 1])
def test_prompt_nonfinite_sequences_next_to_finite_ones(cuda, dtype, d, kernel):
    """Every second of 36 sequences holds NaN and infinities; the others' outputs and weights are theirs alone."""
    S, B = lib(), 36
    r = np.random.default_rng(d)
    lens, old = r.integers(1, 140, B), r.integers(0, 90, B)
    p = Prompt(S, dtype, d, 2, 1, lens.tolist(), (lens + old).tolist(), seed=19, kernel=kernel)
    for b in range(1, B, 2):
        p.qb[p.cu_q[b]:p.cu_q[b + 1]] = float("inf")
        p.kb[p.cu_kv[b]:p.cu_kv[b + 1]] = float("nan")
        p.vb[p.cu_kv[b]:p.cu_kv[b + 1]] = float("-inf")
    p.run()
    q, k, v = host(p.q), host(p.k), host(p.v)
    for b in range(0, B, 2):
        rows, keys = slice(p.cu_q[b], p.cu_q[b + 1]), slice(p.cu_kv[b], p.cu_kv[b + 1])
        n_q, n = p.cu_q[b + 1] - p.cu_q[b], p.cu_kv[b + 1] - p.cu_kv[b]
        ref, w = R.prompt_attention(q[rows], k[keys], v[keys], [0, n_q], [0, n], p.n_w)
        spread, _ = R.prompt_attention(q[rows], k[keys], np.abs(v[keys]), [0, n_q], [0, n], p.n_w)
        e = score_step(q[rows], k[keys], n)
        check_out(host(p.o)[rows], ref, spread, e, dtype, UBF if dtype == BF and kernel == 0 else 0.0, f"sequence {b}")
        check_weight(host(p.w)[b], host(p.w0)[b], w[0], e, f"sequence {b}")
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("H,Hk,lens,kv", [
    (2, 2, [5], [2500]), (6, 2, [1], [1025]), (3, 1, [300], [5000]), (4, 2, [40, 1, 0, 130], [900, 2900, 2000, 131]),
    (2, 1, [2, 20, 9], [6000, 10, 0])])
def test_prompt_few_rows_over_long_histories(cuda, dtype, d, H, Hk, lens, kv):
    """The keys of a row tile may be split over CTAs: ends inside a tile, splits without keys, sequences without any."""
    Prompt(lib(), dtype, d, H, Hk, lens, kv, seed=20, front=2, back=3).run().check(UBF if dtype == BF else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_split_without_weights_repeats_its_bits(cuda, dtype):
    S = lib()
    p = Prompt(S, dtype, 64, 4, 4, [7, 30], [4000, 3000], seed=21)
    a = S.make_prompt_args(p.q, p.k, p.v, p.o, i32(p.cu_q), i32(p.cu_kv), dev_status=p.status)
    nb = S.prompt_workspace_size(a)
    first = None
    for fill in (0, 255, 127):      # whatever the workspace held
        p.o.fill_(7)
        w = torch.full((nb + 256,), fill, dtype=torch.uint8, device="cuda")
        S.prompt_attention(a, w, nb)
        torch.cuda.synchronize()
        assert (w[nb:] == fill).all()
        first = p.o.clone() if first is None else first
        assert torch.equal(first, p.o)
    ref, _ = R.prompt_attention(host(p.q), host(p.k), host(p.v), p.cu_q, p.cu_kv, 1)
    spread, _ = R.prompt_attention(host(p.q), host(p.k), np.abs(host(p.v)), p.cu_q, p.cu_kv, 1)
    check_out(host(p.o), ref, spread, score_step(host(p.q), host(p.k), 4000), dtype, UBF if dtype == BF else 0.0)
