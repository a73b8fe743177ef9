"""The dense half of a batched decode block on the GPU against the fp64 oracle
(oracle/block.py): norm with 8-bit rows, 8-bit product, appending to and reading
the paged 4-bit cache, attention over it, and a run of them around the sparse FFN.

Tolerances.  A rounding to a type is at most half a step: eps/2 of the value (fp16
2^-11, bf16 2^-8, fp32 2^-24).  Each bar below counts the roundings of its path.
"""
import math

import numpy as np
import pytest

import activation_sparse_ffn_predictor_b200 as sp
import oracle as O
import oracle.block as OB

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half a step among the subnormals
F32 = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dtype)


def within(got, want, bar, what=""):
    got, want, bar = np.broadcast_arrays(np.asarray(got, np.float64), want, bar)
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), "%s: %d of %d beyond the bar, e.g. %s" % (
        what, bad.sum(), bad.size, [tuple(float(x) for x in v) for v in zip(got[bad][:3], want[bad][:3], bar[bad][:3])])


# ------------------------------------------------------------------------------------ norm_quant
def check_norm(x, y, g, eps, x_out, q, scale, dtype):
    T, d = x.shape
    u, w, s = OB.norm_quant(f64(x), None if y is None else f64(y), None if g is None else f64(g), eps)
    # w 127 / a: u, w and a (two roundings each) and the quotient and product, six in all, of numbers up to 127
    within(f64(q), w, 0.5 + 127 * 6 * F32, "q")
    # the row's maximum 2, the sum of squares' chain of additions (halved by the root), root, quotient, product
    within(f64(scale), s, s * (d / 256 / 2 + 16) * F32, "scale")
    if x_out is not None:
        within(f64(x_out), u, np.abs(u) * (HALF[dtype] + 2 * F32) + TINY[dtype], "x_out")
    # the definition in fp32, bit for bit
    f = np.float32
    uf = f64(x).astype(f) + (f(0) if y is None else f64(y).astype(f))
    wf = uf if g is None else uf * f64(g).astype(f)
    a = np.abs(wf).max(axis=1, keepdims=True)
    r = np.divide(f(127), a, out=np.zeros_like(a), where=a > 2.0 ** -119)
    assert np.array_equal(q.cpu().numpy(), np.clip(np.rint(wf * r), -127, 127).astype(np.int8))


@pytest.mark.parametrize("d", [1, 7, 64, 96, 1000, 1024, 1032, 4096, 5120, 7168, 9216, 9217, 16384])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm_quant(d, dtype):
    for T, ykind, gain in ((1, "f32", True), (5, "same", True), (33, "none", False), (3, "f32", False)):
        gen = torch.Generator(device="cuda").manual_seed(d + T)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        x, g = (3 * n(T, d)).to(DT[dtype]), (1 + 0.3 * n(d)).to(DT[dtype]) if gain else None
        y = None if ykind == "none" else n(T, d).to(torch.float32 if ykind == "f32" else DT[dtype])
        xo, q, s = torch.empty_like(x), torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        sp.norm_quant(x, y, g, xo, q, s, eps=1e-5)
        check_norm(x, y, g, 1e-5, xo, q, s, dtype)
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        sp.norm_quant(x, y, g, None, q2, s2, eps=1e-5)           # without the sum, and the same bits again
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("d,pad,shift", [(64, 8, 8), (100, 3, 1), (1024, 1, 0), (1024, 8, 4), (4100, 12, 2), (9216, 16, 16)])
def test_norm_quant_strides_in_place_and_what_lies_between_rows(d, pad, shift):
    """Padded rows at shifted addresses, x_out on x; the bytes between the rows stay."""
    T, gen = 6, torch.Generator(device="cuda").manual_seed(9)

    def rows(dtype, fill):
        whole = torch.full((T * (d + pad) + shift,), fill, dtype=dtype, device="cuda")
        return whole, whole[shift:].view(T, d + pad)[:, :d]

    wx, x = rows(torch.bfloat16, 7.0)
    x.copy_(torch.randn(T, d, generator=gen, device="cuda"))
    wy, y = rows(torch.float32, 7.0)
    y.copy_(torch.randn(T, d, generator=gen, device="cuda"))
    wq, q = rows(torch.int8, 99)
    s, before = torch.empty(T, device="cuda"), x.clone()
    sp.norm_quant(x, y, None, x, q, s)
    check_norm(before, y, None, 1e-6, x, q, s, "bf16")
    for whole, fill in ((wx, 7.0), (wq, 99)):
        gaps = whole[shift:].view(T, d + pad)[:, d:]
        assert (gaps == fill).all() and (whole[:shift] == fill).all()


@pytest.mark.parametrize("d", [96, 501, 1024, 4096, 9216])
def test_norm_quant_sum_in_place_of_the_addend(d):
    """x_out is y, of the storage type and the same stride."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    x, y = (torch.randn(7, d, generator=gen, device="cuda").to(torch.float16) for _ in range(2))
    q, s, before = torch.empty(7, d, dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda"), y.clone()
    sp.norm_quant(x, y, None, y, q, s)
    check_norm(x, before, None, 1e-6, y, q, s, "f16")


def test_norm_quant_special_rows():
    d = 512
    x = torch.randn(9, d, device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[1, 5], x[2, 7], x[3, 9] = math.inf, -math.inf, math.nan
    x[4] = 1e-38                       # below the smallest row that has a factor
    x[5] = 3e38                        # the sum of squares leaves fp32
    x[6] *= 1e15
    x[7] *= 1e-15
    for d0 in (d, 500 + 1):            # the wide path and the other one
        v = x[:, :d0].contiguous()
        q, s, xo = torch.full((9, d0), 5, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda"), torch.empty_like(v)
        sp.norm_quant(v, None, None, xo, q, s)
        assert torch.equal(xo[:1], v[:1]) and torch.equal(xo[4:], v[4:])
        assert (q[:6] == 0).all() and s[0] == 0 and s[4] == 0 and torch.isnan(s[[1, 2, 3, 5]]).all()
        check_norm(v[6:], None, None, 1e-6, xo[6:], q[6:], s[6:], "bf16")


@pytest.mark.parametrize("d", [256, 501, 4096, 8192, 9216])      # every form of the wide path, and the other one
@pytest.mark.parametrize("gain", [math.nan, math.inf, -math.inf])
def test_norm_quant_gain_that_is_not_finite(d, gain):
    """One channel's gain is not a number, or infinite: no row has a maximum, also where the channel itself holds 0."""
    x = torch.randn(5, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d)).to(torch.bfloat16)
    at = d // 3
    x[1:4, at] = 0
    x[3] = 0
    g = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    g[at] = gain
    y = torch.zeros(5, d, device="cuda")
    q, s, xo = torch.full((5, d), 5, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda"), torch.empty_like(x)
    sp.norm_quant(x, y, g, xo, q, s)
    assert torch.isnan(s).all() and (q == 0).all() and torch.equal(xo, x)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d", [1, 33, 256, 9216, 20001, 131072])
def test_quantize_rows(d, dtype):
    T = 4
    x = torch.randn(T, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d)).to(DT.get(dtype, torch.float32))
    x[2] = 0
    q, s = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    sp.quantize_rows(x, q, s)
    v = f64(x)
    a = np.abs(v).max(axis=1, keepdims=True)
    within(f64(q), np.divide(127 * v, a, out=np.zeros_like(v), where=a > 0), 0.5 + 127 * 3 * F32)
    within(f64(s), a[:, 0] / 127, a[:, 0] / 127 * F32 * 2)
    x[1, d // 2], x[3, 0] = math.nan, math.inf
    sp.quantize_rows(x, q, s)
    assert torch.isnan(s[[1, 3]]).all() and (q[[1, 3]] == 0).all() and s[0] > 0


# --------------------------------------------------------------------------------------- Linear8
def mm8_data(T, K, N, dtype, bias, seed, full=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randint(-128 if full else -127, 128, s, generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    A, W = r(T, K), r(N, K)
    sa, sw = torch.rand(T, generator=gen, device="cuda") + 0.1, (torch.rand(N, generator=gen, device="cuda") + 0.1) / (8000 * math.sqrt(K))
    b = torch.randn(N, generator=gen, device="cuda").to(DT[dtype]) if bias else None
    return A, W, sa, sw, b


def check_mm8(y, A, W, sa, sw, b, dtype):
    want = OB.mm8(A.cpu().numpy(), W.cpu().numpy(), f64(sa), f64(sw), None if b is None else f64(b))
    size = np.abs(want) + 2 * (0 if b is None else np.abs(f64(b)))      # |product| <= |y| + |bias|
    # the sum to fp32, the scales' product, their product, the bias: four roundings in fp32, then one to the type
    within(f64(y), want, np.abs(want) * HALF[dtype] * (1 + 2.0 ** -10) + 5 * F32 * size + TINY[dtype], "y")


@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 4096, 1000), (2, 48, 129), (3, 1040, 64), (15, 512, 130), (16, 9216, 256), (17, 2064, 513),
                                   (32, 7168, 1024), (33, 64, 5000), (64, 16384, 96), (100, 272, 777), (128, 1024, 2048), (129, 4096, 640),
                                   (256, 5120, 1280), (300, 1008, 384), (1000, 528, 1100), (2048, 256, 260)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear8(T, K, N, dtype):
    A, W, sa, sw, b = mm8_data(T, K, N, dtype, T % 2 == 1, T + K + N)
    lin = sp.Linear8(W, sw, b, max_tokens=T + 5, dtype=DT[dtype])
    y = torch.full((T, N), math.nan, dtype=DT[dtype], device="cuda")
    lin.forward(A, sa, y)
    check_mm8(y, A, W, sa, sw, b, dtype)
    y2 = torch.zeros_like(y)
    lin.forward(A, sa, y2)
    assert torch.equal(y, y2)
    assert lin.last_device_error() == (sp.OK, 0)


def test_linear8_largest_sums_are_exact():
    """All products 2^14 over the widest K: the sum is 2^31 - a little below what 32 bits hold."""
    K, N, T = 131072, 40, 3
    A, W = torch.full((T, K), -128, dtype=torch.int8, device="cuda"), torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    A[:, -1] = -127                                  # 2^31 - 128
    W[1] = 127                                       # and the most negative row
    sa, sw = torch.ones(T, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    sp.Linear8(W, sw, None, max_tokens=T, dtype=torch.float16).forward(A, sa, y)
    check_mm8(y, A, W, sa, sw, None, "f16")


@pytest.mark.parametrize("T,K,N", [
    # one CTA a tile: a line of cut tiles, two or three of them in a share; equal rounds, the last not full; whole tiles
    # before the line; several token tiles
    (32, 400, 128 * 170), (1, 272, 128 * 295 - 7), (48, 272, 128 * 300), (280, 272, 128 * 80 - 50), (250, 272, 100),
    (176, 400, 128 * 170 - 3), (350, 272, 128 * 90),
    # pairs of CTAs: the same
    (256, 400, 256 * 84 - 3), (256, 144, 256 * 140 - 9), (256, 272, 256 * 160), (700, 272, 256 * 28 + 9), (5000, 144, 1408)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear8_more_tiles_than_ctas(T, K, N, dtype):
    """Every CTA goes through several tiles: the ring, both accumulators and the scales go from one to the next."""
    A, W, sa, sw, b = mm8_data(T, K, N, dtype, True, T + K + N)
    lin = sp.Linear8(W, sw, b, max_tokens=T, dtype=DT[dtype])
    y, y2 = (torch.full((T, N), math.nan, dtype=DT[dtype], device="cuda") for _ in range(2))
    lin.forward(A, sa, y)
    check_mm8(y, A, W, sa, sw, b, dtype)
    for _ in range(3):
        lin.forward(A, sa, y2)
        assert torch.equal(y, y2)
    assert lin.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("T,N", [(3, 40), (200, 300)])
def test_linear8_sum_of_two_to_the_31(T, N):
    """The one sum that 32 bits with a sign do not hold: 131,072 products of -128 and -128."""
    K = 131072
    A, W = torch.full((T, K), -128, dtype=torch.int8, device="cuda"), torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    A[1], W[1] = 127, 127                            # beside it the most negative sums, and sums next to it
    A[2, 77] = -127
    sa, sw = torch.ones(T, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    sp.Linear8(W, sw, None, max_tokens=T, dtype=torch.float16).forward(A, sa, y)
    check_mm8(y, A, W, sa, sw, None, "f16")
    assert y[0, 0] == 2048


def test_linear8_strides_streams_and_what_lies_beyond():
    T, K, N = 21, 1024, 1500
    A, W, sa, sw, b = mm8_data(T, K, N, "bf16", True, 5, full=True)
    wideA = torch.full((T, K + 32), 77, dtype=torch.int8, device="cuda")
    wideA[:, :K] = A
    out = torch.full((T + 4, N + 6), 3.0, dtype=torch.bfloat16, device="cuda")
    lin = sp.Linear8(W, sw, b, max_tokens=64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lin.forward(wideA[:, :K], sa, out[:T, :N], stream=st)
    st.synchronize()
    check_mm8(out[:T, :N], A, W, sa, sw, b, "bf16")
    assert (out[T:] == 3).all() and (out[:, N:] == 3).all()
    odd = torch.zeros(T * (N + 1) + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, N + 1)[:, :N]   # rows of any alignment
    lin.forward(A, sa, odd)
    assert torch.equal(odd, out[:T, :N])
    lin.forward(A[:0], sa[:0], out[:0, :N])
    nan = sa.clone()
    nan[4] = math.nan                                # a row that could not be quantised shows
    lin.forward(A, nan, odd)
    assert torch.isnan(odd[4]).all() and torch.equal(odd[5:], out[5:T, :N])


def test_contexts_are_ready_for_any_stream():
    """Made while the current stream is busy, used at once on another one: the workspace is clean by then."""
    T, K, N = 8, 4096, 3000
    A, W, sa, sw, b = mm8_data(T, K, N, "f16", True, 61)
    y = torch.full((T, N), math.nan, dtype=torch.float16, device="cuda")
    page, n = 16, 40
    lens, table = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    x, big = torch.randn(1, 2, 64, device="cuda").half(), torch.randn(8192, 8192, device="cuda")
    K4, V4 = (torch.empty(3, page, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    makes = (lambda: sp.Linear8(W, sw, b, max_tokens=T), lambda: sp.KvCache4(3, page, 2, 2, 64, torch.float16, 1, 1))
    side, made = torch.cuda.Stream(), []
    for make, use in zip(makes, (lambda c: c.forward(A, sa, y, stream=side), lambda c: c.append(None, x, x, table, lens, None, stream=side))):
        first = make()
        use(first)                                # the first launch of a kernel may wait for the device
        torch.cuda.synchronize()
        if not made:
            y.fill_(math.nan)
        sizes = [t.numel() for t in (getattr(first, "pool", x), first.workspace)]
        del first
        dirty = [torch.full((n_bytes,), 255, dtype=torch.uint8, device="cuda") for n_bytes in sizes]
        torch.cuda.synchronize()
        del dirty                                 # what the allocator hands out next is not clean
        for _ in range(20):
            big @ big
        made.append(make())
        use(made[-1])
    lin, cache = made
    cache.read(table[0], K4, V4, stream=side)
    side.synchronize()
    check_mm8(y, A, W, sa, sw, b, "f16")
    assert lin.last_device_error(side) == (sp.OK, 0) and cache.last_device_error(side) == (sp.OK, 0)
    V4 = V4.view(-1, 2, 64)
    # half a step: 32 values of N(0, 1) lie within 8 of one another
    assert (V4[:n - 1] == 0).all() and (V4[n:] == 0).all() and (V4[n - 1] - x[0]).abs().max() < 0.3


def test_linear8_graph_replays_on_new_inputs():
    T, K, N = 8, 2048, 3000
    A, W, sa, sw, b = mm8_data(T, K, N, "f16", True, 6)
    lin, y = sp.Linear8(W, sw, b, max_tokens=T), torch.empty(T, N, dtype=torch.float16, device="cuda")
    lin.forward(A, sa, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.forward(A, sa, y)
        lin.forward(A, sa, y)
    for seed in (7, 8):
        A2, _, sa2, _, _ = mm8_data(T, K, N, "f16", False, seed)
        A.copy_(A2)
        sa.copy_(sa2)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_mm8(y, A, W, sa, sw, b, "f16")


# -------------------------------------------------------------------------------------- KvCache4
class Paged:
    """A pool with scattered pages and a batch of sequences over it."""

    def __init__(self, lens, new, nh, kvh, dh, page, dtype, seed=0, rope=None, spare=2, pad_rows=0):
        r = np.random.default_rng(seed)
        self.r, self.page, self.nh, self.kvh, self.dh, self.dtype = r, page, nh, kvh, dh, dtype
        self.lens, self.new, self.B, self.T = list(lens), list(new), len(lens), sum(new) + pad_rows
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = r.permutation(self.pages)
        self.table = np.full((self.B, max(max(need), 1) + 1), 2 ** 30, np.int32)     # unused entries name no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.freqs, self.inter, self.amp = rope if rope else (np.zeros(0), False, 1.0)
        self.cache = sp.KvCache4(self.pages, page, nh, kvh, dh, DT[dtype], max_seqs=max(self.B, 1), max_tokens=max(self.T, 1),
                                 rope=sp.Rope(self.freqs, self.inter, self.amp) if rope else None)
        self.gtable, self.glens, self.gstart = dev(self.table), dev(np.array(self.lens, np.int32)), dev(self.start)

    def rows(self, heads, scale=1.0):
        return dev(self.r.normal(size=(self.T, heads, self.dh)) * scale).to(DT[self.dtype])

    def fill(self, k_scale=1.0, v_scale=1.0, nan_behind=True):
        """Random cache contents; every token that no sequence covers holds NaN steps and zeros."""
        shape = (self.pages, self.page, self.kvh, self.dh)
        K, V = (OB.quantise((self.r.normal(size=shape) * s).astype(np.float32)) for s in (k_scale, v_scale))
        if nan_behind:
            seen = np.zeros((self.pages, self.page), bool)
            for b, n in enumerate(self.lens):
                for p in range(n):
                    seen[self.table[b, p // self.page], p % self.page] = True
            for _, step, zero in (K, V):
                step[~seen], zero[~seen] = np.nan, np.inf
        self.K, self.V = K, V
        self.cache.pool.copy_(dev(OB.write_pool(K, V, self.page, self.kvh, self.dh).reshape(-1)))

    def of_sequence(self, b, which):
        codes, step, zero = which
        p = np.arange(self.lens[b])
        at = self.table[b, p // self.page], p % self.page
        return OB.values(codes[at], step[at], zero[at]), 15 * step[at].astype(np.float64) + np.abs(zero[at].astype(np.float64))

    def check_attend(self, q, out, scale=None, skip=()):
        scale = self.dh ** -0.5 if scale is None else scale
        G, q, out = self.nh // self.kvh, f64(q), f64(out)
        for b in range(self.B):
            if b in skip or not self.new[b]:
                continue
            K, Kw = self.of_sequence(b, self.K)
            V, Vw = self.of_sequence(b, self.V)
            r0, n, m = int(self.start[b]), self.new[b], self.lens[b]
            vis = np.repeat(np.arange(m)[None, :] <= np.arange(m - n, m)[:, None], G, axis=0)
            for h in range(self.kvh):
                rows = q[r0:r0 + n, h * G:(h + 1) * G].reshape(n * G, self.dh)
                o, p = OB.attend(rows, K[:, h], V[:, h], vis, scale)
                got = out[r0:r0 + n, h * G:(h + 1) * G].reshape(n * G, self.dh)
                # scores: fp32 sums over dh products of |q| (15 step + |zero|), then the exponential's own 2^-22
                ds = np.abs(scale) * (np.abs(rows).sum(1) * Kw[:, h].max(initial=0)) * (self.dh + 16) * F32 + 2.0 ** -21
                # probabilities enter the second product in fp16, once by themselves and once times the step: a
                # rounding each, on numbers as large as 15 step + |zero|
                wide = np.repeat(Vw[:, h].max(axis=0, initial=0), 32)[None, :]
                bar = (2 * HALF["f16"] + 2 * ds[:, None] + 2.0 ** -18) * wide + HALF[self.dtype] * np.abs(o) + TINY[self.dtype]
                within(got, o, bar, "sequence %d, kv head %d" % (b, h))


GEOM = [(1, 1, 64, 16), (8, 8, 128, 32), (8, 2, 64, 16), (14, 2, 128, 64), (16, 1, 128, 128), (5, 5, 256, 16), (64, 1, 64, 256), (24, 2, 256, 64)]


@pytest.mark.parametrize("nh,kvh,dh,page", GEOM)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_one_token_each(nh, kvh, dh, page, dtype):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 129, 300, 511, 777]
    c = Paged(lens, [1] * len(lens), nh, kvh, dh, page, dtype, seed=nh + dh)
    c.fill()
    q = c.rows(nh, 2.0)
    out, out2 = torch.full_like(q, math.nan), torch.full_like(q, math.nan)
    c.cache.attend(q, c.gtable, c.glens, None, out)
    c.check_attend(q, out)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out2)       # the same batch with its starts spelled out
    assert torch.equal(out, out2)
    assert c.cache.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("nh,kvh,dh,page", GEOM)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_several_tokens_each(nh, kvh, dh, page, dtype):
    """Drafted tokens, prompts from nothing, sequences without new tokens, rows behind the last."""
    lens, new = [5, 40, 200, 7, 0, 65, 33], [5, 3, 20, 0, 0, 1, 33]
    c = Paged(lens, new, nh, kvh, dh, page, dtype, seed=nh + dh + 1, pad_rows=3)
    c.fill()
    q = c.rows(nh, 2.0)
    q[-3:] = math.nan
    out = torch.full_like(q, 9.0)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out)
    assert (out[-3:] == 9).all()
    assert c.cache.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("nh,kvh,dh,n,length", [(8, 1, 128, 1, 20011), (4, 4, 64, 1, 5000), (32, 8, 128, 1, 9000), (2, 2, 256, 3, 7001),
                                                (8, 8, 64, 100, 1500), (16, 2, 128, 40, 2500)])
def test_attend_long_and_split(nh, kvh, dh, n, length):
    """One sequence whose keys are split over many blocks; a second, short one beside it."""
    c = Paged([length, 3], [n, 1], nh, kvh, dh, 64, "f16", seed=n)
    c.fill()
    q = c.rows(nh, 3.0)
    out, out2 = torch.full_like(q, math.nan), torch.full_like(q, math.nan)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out)
    for _ in range(3):                      # the order of sums is fixed: the same bits
        c.cache.attend(q, c.gtable, c.glens, c.gstart, out2)
        assert torch.equal(out, out2)


@pytest.mark.parametrize("nh,kvh,dh,page,n,length", [(4, 1, 128, 64, 1500, 1500), (8, 2, 64, 16, 700, 3001), (2, 2, 256, 32, 300, 1000),
                                                     (16, 2, 128, 32, 513, 514), (64, 1, 64, 256, 200, 1100)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_prompts(nh, kvh, dh, page, n, length, dtype):
    """Hundreds of new tokens of one sequence, from nothing or over what is cached of it, beside a decoded one."""
    c = Paged([length, 77], [n, 1], nh, kvh, dh, page, dtype, seed=n)
    c.fill()
    q = c.rows(nh, 2.0)
    out = torch.full_like(q, math.nan)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out)
    assert c.cache.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("case", ["large-q", "tiny-q", "zero-q", "large-v", "tiny-v", "mixed-v", "sharp", "scale-0", "scale-negative"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_ranges(case, dtype):
    c = Paged([300, 17, 1], [1, 2, 1], 8, 2, 128, 16, dtype, seed=5)
    big = {"large-v": 2000.0, "tiny-v": 1e-4}.get(case, 1.0)
    c.fill(v_scale=big, k_scale=0.01 if case == "large-q" else 1.0)
    if case == "mixed-v":                   # tokens of very different size side by side
        codes, step, zero = c.V
        f = np.float16(2.0) ** c.r.integers(-10, 8, size=step.shape[:3] + (1,)).astype(np.float16)
        c.V = (codes, (step * f).astype(np.float16), (zero * f).astype(np.float16))
        c.cache.pool.copy_(dev(OB.write_pool(c.K, c.V, c.page, c.kvh, c.dh).reshape(-1)))
    q = c.rows(8, {"large-q": 3e4 if dtype == "bf16" else 3000.0, "tiny-q": 1e-6, "sharp": 12.0}.get(case, 1.0))
    if case == "zero-q":
        q.zero_()
    scale = {"large-q": 1e-4, "scale-0": 0.0, "scale-negative": -0.05}.get(case)
    out = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out, scale=scale)
    c.check_attend(q, out, scale=scale)


@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_values_with_a_mean_far_above_their_spread(dtype, dh):
    """V around 4 with a spread of 0.01: nearly all of the output comes from the zeros."""
    c = Paged([1, 2, 3, 4, 7, 33, 300], [1, 1, 2, 1, 1, 3, 1], 4, 2, dh, 16, dtype, seed=17)
    c.fill(v_scale=0.01)
    c.V = c.V[0], c.V[1], (c.V[2] + np.float16(4)).astype(np.float16)
    c.cache.pool.copy_(dev(OB.write_pool(c.K, c.V, c.page, c.kvh, c.dh).reshape(-1)))
    q = c.rows(4, 0.03)
    out = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    step = np.nanmax(c.V[1].astype(np.float64))
    for b in range(c.B):
        K, Kw = c.of_sequence(b, c.K)
        V, Vw = c.of_sequence(b, c.V)
        r0, n, m = int(c.start[b]), c.new[b], c.lens[b]
        vis = np.repeat(np.arange(m)[None, :] <= np.arange(m - n, m)[:, None], 2, axis=0)
        for h in range(2):
            rows = f64(q)[r0:r0 + n, 2 * h:2 * h + 2].reshape(2 * n, dh)
            o, _ = OB.attend(rows, K[:, h], V[:, h], vis, dh ** -0.5)
            # scores as in check_attend.  fp16: p s rounded once, codes around 8 at most 8 of them; bf16: a rounding of
            # p on the whole value and one of p s on 15 steps
            ds = dh ** -0.5 * np.abs(rows).sum(1) * Kw[:, h].max() * (dh + 16) * F32 + 2.0 ** -21
            own = HALF["f16"] * (8 * step if dtype == "f16" else Vw.max() + 15 * step)
            bar = (2 * ds[:, None] + 2.0 ** -18) * Vw.max() + own + HALF[dtype] * np.abs(o)
            within(f64(out)[r0:r0 + n, 2 * h:2 * h + 2].reshape(2 * n, dh), o, bar, "sequence %d" % b)


@pytest.mark.parametrize("nh,kvh,dh,page", GEOM)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_steps_that_grow_along_a_sequence(nh, kvh, dh, page, dtype):
    """V grows by 2^16 from the first position to the last, each group of dims at a level of its own, or falls as much."""
    c = Paged([300, 77, 300, 40], [1, 5, 2, 40], nh, kvh, dh, page, dtype, seed=nh + dh + 3)
    c.fill()
    level = np.zeros(c.V[1].shape, np.int64)
    for b, n in enumerate(c.lens):
        p = np.arange(n)
        e = (-9 + 16 * (p if b != 2 else n - 1 - p) // n)[:, None, None] + (np.arange(dh // 32) * 5 % 7 - 3)
        level[c.table[b, p // page], p % page] = e
    f = np.exp2(level).astype(np.float16)
    c.V = c.V[0], (c.V[1] * f).astype(np.float16), (c.V[2] * f).astype(np.float16)
    c.cache.pool.copy_(dev(OB.write_pool(c.K, c.V, page, kvh, dh).reshape(-1)))
    q = c.rows(nh, 2.0)
    out = torch.full_like(q, math.nan)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out)


@pytest.mark.parametrize("n,G", [(1, 1), (3, 4)])
@pytest.mark.parametrize("v", ["1e-1", "1e-2", "1e-3", "1e-4", "neighbours", "groups"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_one_key_stands_out_of_many_small_values(dtype, v, n, G):
    """1800 sequences over the same 100,003 positions, so that one warp walks tens of thousands of them: one key has most
    of the weight, each of the others some 1e-6 of it.  V is small as a whole, or differs by 2^10 between neighbouring
    tokens, or by 2^12 between groups of dims."""
    L, kvh, dh, page, B = 100003, 1, 128, 64, 1800
    c = Paged([L], [n], G * kvh, kvh, dh, page, dtype, seed=n + len(v))
    c.fill(v_scale=float(v) if v[0] == "1" else 0.1)
    at = c.table[0, 5000 // page], 5000 % page
    codes, step, zero = c.K                       # the first 32 dims hold nothing but the one key's mark
    codes[..., :32], step[..., 0], zero[..., 0] = 0, 0, 0
    zero[at[0], at[1], :, 0] = 4.9                # scale 32 4.9 = 13.9: e^13.9 beside 100,003 times e^0.5
    if v[0] != "1":
        step, zero = c.V[1].copy(), c.V[2].copy()
        small = (slice(None), slice(1, None, 2)) if v == "neighbours" else (slice(None),) * 3 + (1,)
        for a in (step, zero):
            a[small] = a[small] * np.float16(2.0 ** (-10 if v == "neighbours" else -12))
        c.V = c.V[0], step, zero
    c.cache.pool.copy_(dev(OB.write_pool(c.K, c.V, page, kvh, dh).reshape(-1)))
    many = sp.KvCache4(c.pages, page, G * kvh, kvh, dh, DT[dtype], max_seqs=B, max_tokens=B * n, pool=c.cache.pool)
    q = dev(c.r.normal(size=(B * n, G * kvh, dh))).to(DT[dtype])
    q[..., :32] = 1
    out = torch.full_like(q, math.nan)
    start = dev(np.arange(B + 1, dtype=np.int32) * n)
    many.attend(q, c.gtable.expand(B, -1).contiguous(), c.glens.expand(B).contiguous(), start, out)
    for b in (0, B // 2, B - 1):
        c.check_attend(q[b * n:(b + 1) * n], out[b * n:(b + 1) * n])


def test_attend_rows_that_are_not_numbers_stay_alone():
    c = Paged([40, 50], [2, 1], 4, 2, 64, 16, "f16", seed=6)
    c.fill()
    q = c.rows(4)
    good = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, good)
    q[1, 2, 5] = math.nan
    q[2, 0, 0] = math.inf
    out = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 0]).all()
    ok = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    ok[1, 2] = ok[2, 0] = False
    assert torch.equal(out[ok], good[ok])


@pytest.mark.parametrize("dh,page,G", [(64, 16, 1), (64, 64, 8), (128, 64, 2), (128, 16, 4), (256, 32, 1), (256, 64, 5)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_values_that_are_not_finite_reach_only_rows_that_see_them(dtype, dh, page, G):
    """The last drafted token's key or value holds a NaN or an infinity: the tokens before it do not see it, though they
    lie in the same tile."""
    c = Paged([40, 71], [1, 3], 2 * G, 2, dh, page, dtype, seed=18)
    c.fill(nan_behind=False)
    q = c.rows(2 * G)
    good = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, good)
    c.check_attend(q, good)
    clean = c.cache.pool.clone()
    at = (c.table[1, 70 // page], 70 % page, 1)            # of the second kv head
    for which, part, bad in (("V", 1, np.nan), ("V", 1, np.inf), ("V", 1, -np.inf), ("V", 2, np.nan), ("V", 2, np.inf), ("V", 2, -np.inf),
                             ("K", 1, np.nan), ("K", 2, np.nan)):
        for g in (0, dh // 32 - 1):
            K, V = (tuple(a.copy() for a in x) for x in (c.K, c.V))
            (K if which == "K" else V)[part][at + (g,)] = bad
            c.cache.pool.copy_(dev(OB.write_pool(K, V, page, 2, dh).reshape(-1)))
            out = torch.empty_like(q)
            c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
            assert torch.isnan(out[3, G:]).all(), (which, part, bad, g)
            out[3, G:] = good[3, G:]
            c.check_attend(q, out)
    c.cache.pool.copy_(clean)
    assert c.cache.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("dh,page", [(64, 16), (128, 64), (256, 32)])
def test_attend_batches_that_are_refused_on_the_device(dh, page):
    """Bad rows, lengths and pages: nothing out of range is touched, the rest of the batch is right, the error is latched."""
    def fresh():
        c = Paged([70, 100, 9], [2, 1, 3], 4, 2, dh, page, "bf16", seed=7)
        c.fill()
        q = c.rows(4)
        return c, q, torch.full_like(q, 5.0)

    c, q, out = fresh()
    c.glens[1] = 10 ** 9                                   # above the table's reach
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out, skip=(1,))
    assert (out[2] == 0).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK
    assert c.cache.last_device_error() == (sp.OK, 0)       # read and cleared

    c, q, out = fresh()
    c.glens[2] = 2                                         # fewer than its three new tokens
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out, skip=(2,))
    assert (out[3:] == 0).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK

    c, q, out = fresh()
    c.glens[0] = -4
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out, skip=(0,))
    assert (out[:2] == 0).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK

    c, q, out = fresh()
    c.gstart[3] = 2 ** 31 - 1                              # rows past the end
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out, skip=(2,))
    assert (out[3:] == 5).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK

    for page_id in (-1, 2 ** 30, c.pages):
        c, q, out = fresh()
        col = 0 if page <= 32 else 1
        c.gtable[1, col] = page_id                         # its tokens are left out
        c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
        c.check_attend(q, out, skip=(1,))
        assert c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK
        K, _ = c.of_sequence(1, c.K)
        V, _ = c.of_sequence(1, c.V)
        vis = np.broadcast_to((np.arange(100) // page != col)[None, :], (2, 100))
        for h in range(2):
            o, _ = OB.attend(f64(q)[2, 2 * h:2 * h + 2], K[:, h], V[:, h], vis, dh ** -0.5)
            within(f64(out)[2, 2 * h:2 * h + 2], o, 0.02 + 0.01 * np.abs(o))

    c, q, out = fresh()
    c.gtable[2] = -7                                       # nothing left: zero rows
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    assert (out[3:] == 0).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK


def test_attend_strides_and_streams():
    c = Paged([33, 90, 5], [1, 1, 1], 6, 3, 64, 16, "f16", seed=8)
    c.fill()
    q = c.rows(6)
    want = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, None, want)
    for pad in (8, 3):                                     # rows of any stride, and heads as one row
        wq, wo = torch.full((3, 6 * 64 + pad), 7.0, dtype=torch.float16, device="cuda"), torch.full((3, 6 * 64 + pad), 7.0, dtype=torch.float16, device="cuda")
        wq[:, :384] = q.view(3, 384)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        c.cache.attend(wq[:, :384], c.gtable, c.glens, None, wo[:, :384].view(3, 6, 64) if pad == 8 else wo[:, :384], stream=st)
        st.synchronize()
        assert torch.equal(wo[:, :384].reshape(3, 6, 64), want) and (wo[:, 384:] == 7).all()


def test_attend_shared_pages_and_a_wide_table():
    """Two sequences over the same prefix pages; the table's row stride is wider than its columns."""
    c = Paged([48, 48], [1, 1], 4, 2, 64, 16, "bf16", seed=9)
    c.table[1, :2] = c.table[0, :2]
    c.fill(nan_behind=False)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = dev(c.table)
    q = c.rows(4)
    out = torch.empty_like(q)
    c.cache.attend(q, wide[:, :c.table.shape[1]], c.glens, None, out)
    c.check_attend(q, out)


def test_attend_steps_of_either_sign():
    """The value is code step + zero, whatever the step's sign: a pool that was not filled by append."""
    c = Paged([90, 33], [1, 1], 4, 2, 128, 16, "f16", seed=31)
    c.fill(v_scale=300.0)
    flip = np.where(c.r.random(c.V[1].shape) < 0.5, -1, 1).astype(np.float16)
    c.V = (c.V[0], (c.V[1] * flip).astype(np.float16), c.V[2])
    c.cache.pool.copy_(dev(OB.write_pool(c.K, c.V, c.page, c.kvh, c.dh).reshape(-1)))
    q = c.rows(4, 2.0)
    out = torch.empty_like(q)
    c.cache.attend(q, c.gtable, c.glens, None, out)
    # a rounding of p s and one of p on numbers up to 15 |step| + |zero| (positions behind the sequences hold NaN)
    wide = np.nanmax(np.abs(c.V[1]).astype(np.float64))
    for b in range(2):
        K, _ = c.of_sequence(b, c.K)
        V, _ = c.of_sequence(b, c.V)
        for h in range(2):
            o, _ = OB.attend(f64(q)[b, 2 * h:2 * h + 2], K[:, h], V[:, h], np.ones((2, c.lens[b]), bool), 128 ** -0.5)
            within(f64(out)[b, 2 * h:2 * h + 2], o, 2 * HALF["f16"] * (15 * wide + 2000) + HALF["f16"] * np.abs(o))


def test_attend_empty_and_padded_calls():
    c = Paged([20, 30], [1, 1], 4, 2, 64, 16, "bf16", seed=32, pad_rows=3)
    c.fill()
    q = c.rows(4)
    out = torch.full_like(q, 4.0)
    c.cache.attend(q, c.gtable, c.glens, None, out)            # five rows, two sequences of one token
    c.check_attend(q, out)
    assert (out[2:] == 4).all()
    before = out.clone()
    c.cache.attend(q[:0], c.gtable, c.glens, torch.zeros(3, dtype=torch.int32, device="cuda"), out[:0])
    c.cache.attend(q, c.gtable[:0], c.glens[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), out)
    c.cache.attend(q, c.gtable, c.glens, torch.zeros(3, dtype=torch.int32, device="cuda"), out)      # no new tokens at all
    c.cache.append(q[:0], q[:0, :2], q[:0, :2], c.gtable, c.glens, torch.zeros(3, dtype=torch.int32, device="cuda"), out[:0])
    assert torch.equal(out, before) and c.cache.last_device_error() == (sp.OK, 0)
    c.glens[0] = 2 ** 31 - 1                                   # past what positions may reach
    c.cache.attend(q, c.gtable, c.glens, None, out)
    assert (out[0] == 0).all() and torch.equal(out[1], before[1]) and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK


@pytest.mark.parametrize("B", [33, 200])
def test_attend_many_sequences(B):
    """More sequences than a warp has lanes, some without new tokens, lengths from 1 on."""
    r = np.random.default_rng(B)
    lens = r.integers(1, 90, B).tolist()
    new = [int(x) if r.random() < 0.8 else 0 for x in np.minimum(lens, r.integers(1, 4, B))]
    c = Paged(lens, new, 4, 2, 64, 16, "bf16", seed=B)
    c.fill()
    q = c.rows(4, 2.0)
    out = torch.full_like(q, math.nan)
    c.cache.attend(q, c.gtable, c.glens, c.gstart, out)
    c.check_attend(q, out)


def test_two_contexts_at_once_and_a_graph_beside_eager_calls():
    """Two caches on two streams, and one cache whose captured call is replayed between eager ones on its stream."""
    cs = [Paged([700, 60], [1, 1], 8, 2, 128, 64, "f16", seed=40 + i) for i in range(2)]
    for c in cs:
        c.fill()
    qs = [c.rows(8, 2.0) for c in cs]
    outs, streams = [torch.empty_like(q) for q in qs], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, o, s in zip(cs, qs, outs, streams):
            c.cache.attend(q, c.gtable, c.glens, None, o, stream=s)
    torch.cuda.synchronize()
    for c, q, o in zip(cs, qs, outs):
        c.check_attend(q, o)
    c, q = cs[0], qs[0]
    captured, eager = torch.empty_like(q), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attend(q, c.gtable, c.glens, None, captured)
        c.cache.attend(q, c.gtable, c.glens, None, captured)
    for _ in range(3):
        captured.zero_()
        eager.zero_()
        c.cache.attend(q, c.gtable, c.glens, None, eager)
        g.replay()
        c.cache.attend(q, c.gtable, c.glens, None, eager)
        torch.cuda.synchronize()
        assert torch.equal(captured, outs[0]) and torch.equal(eager, outs[0])


def test_offsets_past_32_bits():
    """Pages whose bytes lie beyond 4 GiB of the pool: appended, attended to and read."""
    kvh, dh, page, pages, n = 8, 128, 64, 56000, 100
    cache = sp.KvCache4(pages, page, kvh, kvh, dh, torch.bfloat16, max_seqs=1, max_tokens=n)
    assert cache.pool.numel() > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(50)
    q, k, v = (torch.randn(n, kvh, dh, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    ids = [pages - 1, pages - 2]
    table, lens = torch.tensor([ids], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cache.append(None, k, v, table, lens, start)
    out = torch.empty_like(q)
    cache.attend(q, table, lens, start, out)
    K, V = (torch.empty(2, page, kvh, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(table[0], K, V)
    whole = cache.pool.view(pages, -1)
    got = OB.read_pool(whole[pages - 2:].flip(0).cpu().numpy(), page, kvh, dh)
    assert (whole[:pages - 2].view(torch.int64).amax() == 0) and cache.last_device_error() == (sp.OK, 0)
    for name, x, t in (("K", k, K), ("V", v, V)):
        codes, step, zero = (a.reshape(2 * page, *a.shape[2:])[:n] for a in got[name])
        for a, b in zip((codes, step, zero), OB.quantise(f64(x).astype(np.float32))):
            assert np.array_equal(a, b)
        want = OB.values(codes, step, zero)
        within(f64(t).reshape(2 * page, kvh, dh)[:n], want, np.abs(want) * (HALF["bf16"] + 2 * F32) + TINY["bf16"])
    c = Paged.__new__(Paged)
    c.page, c.nh, c.kvh, c.dh, c.dtype, c.B = page, kvh, kvh, dh, "bf16", 1
    c.lens, c.new, c.start, c.table = [n], [n], np.array([0, n]), np.array([[0, 1]])
    c.K, c.V = got["K"], got["V"]
    c.check_attend(q, out)


ROPES = {
    "none": None,
    "half": (10000.0 ** (-np.arange(32) / 32), False, 1.0),
    "interleaved": (10000.0 ** (-np.arange(32) / 32), True, 1.0),
    "part-half": (10000.0 ** (-np.arange(9) / 9), False, 1.0),        # 18 of the dims: pairs across 16-byte pieces
    "part-interleaved": (10000.0 ** (-np.arange(5) / 5), True, 1.0),
    "scaled": sp.rope_frequencies(64, 10000.0, "parts", 8.0, 4096.0) if sp else None,
}


@pytest.mark.parametrize("rope", ["none", "half", "interleaved", "part-half", "part-interleaved", "scaled"])
@pytest.mark.parametrize("nh,kvh,dh,page", [(1, 1, 64, 16), (8, 2, 128, 64), (6, 6, 64, 32), (3, 3, 256, 16)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_and_read(rope, nh, kvh, dh, page, dtype):
    r = ROPES[rope]
    if rope == "scaled":
        r = (r[0], False, r[1])
    lens, new = [1, 20, 70, 100000, 9, 16], [1, 3, 33, 2, 0, 16]
    lens = [n if n < 1000 else 700 for n in lens]
    c = Paged(lens, new, nh, kvh, dh, page, dtype, seed=11, rope=r, pad_rows=2)
    c.fill(nan_behind=False)
    before = c.cache.pool.clone()
    q, k, v = c.rows(nh), c.rows(kvh, 3.0), c.rows(kvh)
    k[0, 0, :32] = 0.75                       # a group of one value: step 0
    qo = torch.full_like(q, 9.0)
    c.cache.append(q, k, v, c.gtable, c.glens, c.gstart, qo)
    assert c.cache.last_device_error() == (sp.OK, 0)
    T = sum(new)
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)])
    seq = np.repeat(np.arange(len(new)), new)
    at = (c.table[seq, pos // page], pos % page)
    turn = lambda x: OB.rotate(f64(x)[:T], pos, c.freqs, c.inter, c.amp)  # noqa: E731
    # rotation: cosine and sine (within 2 of fp32's last place, and once more for the amplitude), two products, a sum
    pair = np.sqrt(2.0) * c.amp * np.abs(f64(q)[:T]).max(axis=-1, keepdims=True)
    within(f64(qo)[:T], turn(q), np.abs(turn(q)) * HALF[dtype] + 6 * F32 * pair + TINY[dtype], "q_out")
    assert (qo[T:] == 9).all()
    codes = OB.read_pool(c.cache.pool.cpu().numpy(), page, kvh, dh)
    for name, want in (("K", turn(k)), ("V", f64(v)[:T])):
        if name == "V" or r is None:          # no arithmetic before the quantiser: its fp32 definition, bit for bit
            for got, ref in zip(codes[name], OB.quantise(want.astype(np.float32))):
                assert np.array_equal(got[at], ref), name
        c64, s64, z64 = OB.quantise(want, np.float64)
        got = OB.values(*(a[at] for a in codes[name]))
        step, lo = np.repeat(s64.astype(np.float64), 32, -1), np.abs(np.repeat(z64.astype(np.float64), 32, -1))
        big = np.abs(want).max(axis=-1, keepdims=True)
        # half a step, the fp16 roundings of zero and step at the ends of the range, the rotation's fp32
        within(got, want, step / 2 + 2.0 ** -11 * (lo + 15 * step) + 2.0 ** -23 + 16 * F32 * big, name)
    # every other byte of the pool stays: the same pool with the new places taken from the old
    after = c.cache.pool.clone()
    old = OB.read_pool(before.cpu().numpy(), page, kvh, dh)
    for name in "KV":
        for a, o in zip(codes[name], old[name]):
            a[at] = o[at]
    assert np.array_equal(OB.write_pool(codes["K"], codes["V"], page, kvh, dh).reshape(-1), before.cpu().numpy())
    # read gives code step + zero, rounded once
    ids = torch.randperm(c.pages, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.int32)
    K, V = (torch.empty(c.pages, page, kvh, dh, dtype=DT[dtype], device="cuda") for _ in range(2))
    c.cache.read(ids, K, V)
    now = OB.read_pool(after.cpu().numpy(), page, kvh, dh)
    for t, name in ((K, "K"), (V, "V")):
        want = OB.values(*(a[ids.cpu().numpy()] for a in now[name]))
        within(f64(t), want, np.abs(want) * (HALF[dtype] + 2 * F32) + TINY[dtype], "read " + name)
    # in place, k and v alone, the token at a time: the same bytes
    c.cache.pool.copy_(before)
    c.cache.append(q, k, v, c.gtable, c.glens, c.gstart, q)
    assert torch.equal(c.cache.pool, after) and torch.equal(q[:T], qo[:T])
    c.cache.pool.copy_(before)
    c.cache.append(None, k, v, c.gtable, c.glens, c.gstart)
    assert torch.equal(c.cache.pool, after)


def test_append_far_positions_keep_their_angles():
    """Position 3,000,000 of a short table: only the last page of the table row is looked at."""
    page, far, n = 256, 3_000_000, 4
    width = far // page + 1
    cache = sp.KvCache4(2, page, 1, 1, 64, torch.float16, max_seqs=1, max_tokens=n, rope=sp.Rope(10000.0 ** (-np.arange(32) / 32)))
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    x = torch.randn(n, 1, 64, device="cuda").half()
    qo = torch.empty_like(x)
    lens, start = torch.tensor([far], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cache.append(x, x, x, table, lens, start, qo)
    want = OB.rotate(f64(x), np.arange(far - n, far), 10000.0 ** (-np.arange(32) / 32), False)
    pair = np.sqrt(2.0) * np.abs(f64(x)).max(axis=-1, keepdims=True)
    within(f64(qo), want, np.abs(want) * HALF["f16"] + 6 * F32 * pair + TINY["f16"])
    assert cache.last_device_error() == (sp.OK, 0)


def test_append_strided_rows_of_a_joint_projection():
    for pad in (0, 8, 1):
        nh, kvh, dh, page = 4, 2, 64, 16
        c = Paged([30, 17, 1], [2, 1, 1], nh, kvh, dh, page, "bf16", seed=12, rope=ROPES["half"])
        joint = torch.randn(4, (nh + 2 * kvh) * dh + pad, device="cuda").to(torch.bfloat16)
        q, k, v = joint[:, :nh * dh], joint[:, nh * dh:(nh + kvh) * dh], joint[:, (nh + kvh) * dh:(nh + 2 * kvh) * dh]
        qo = torch.empty(4, nh, dh, dtype=torch.bfloat16, device="cuda")
        c.cache.append(q, k, v, c.gtable, c.glens, c.gstart, qo)
        one = c.cache.pool.clone()
        c.cache.pool.zero_()
        qo2 = torch.empty_like(qo)
        c.cache.append(*(t.contiguous().view(4, -1, dh) for t in (q, k, v)), c.gtable, c.glens, c.gstart, qo2)
        assert torch.equal(one, c.cache.pool) and torch.equal(qo, qo2)


def test_append_special_values_and_refusals_on_the_device():
    nh, kvh, dh, page = 2, 2, 64, 16
    c = Paged([20, 40, 3], [1, 1, 1], nh, kvh, dh, page, "bf16", seed=13)
    k, v = c.rows(kvh), c.rows(kvh)
    k[0, 0, 3], v[1, 1, 40] = math.nan, math.inf
    k[2] = 1e30 * torch.sign(torch.randn_like(k[2].float())).to(torch.bfloat16)       # beyond fp16: held at its largest
    c.cache.append(None, k, v, c.gtable, c.glens, None)
    codes = OB.read_pool(c.cache.pool.cpu().numpy(), page, kvh, dh)
    pos = np.array(c.lens) - 1
    at = (c.table[np.arange(3), pos // page], pos % page)
    ks, vs = codes["K"][1][at], codes["V"][1][at]
    assert np.isnan(ks[0, 0, 0]) and np.isfinite(ks[0, 0, 1]) and np.isnan(vs[1, 1, 1]) and np.isfinite(vs[1, 1, 0])
    assert np.all(np.abs(codes["K"][2][at][2]) == 65504) and np.all(ks[2] == 65504)
    pool = c.cache.pool.clone()
    for lens, table in ((c.glens + 10 ** 6, c.gtable), (c.glens * 0, c.gtable), (c.glens, c.gtable * 0 - 1), (c.glens, c.gtable * 0 + c.pages)):
        c.cache.append(None, c.rows(kvh), c.rows(kvh), table, lens, None)
        assert torch.equal(c.cache.pool, pool) and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK
    bad = torch.tensor([0, 5, -3, 2 ** 30], dtype=torch.int32, device="cuda")         # starts that make no sense
    c.cache.append(None, c.rows(kvh), c.rows(kvh), c.gtable, c.glens, bad)
    assert c.cache.last_device_error()[0] in (sp.OK, sp.ERR_DEVICE_CHECK)
    K = torch.full((2, page, kvh, dh), 4.0, dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    c.cache.read(torch.tensor([c.pages, 0], dtype=torch.int32, device="cuda"), K, V)
    assert (K[0] == 4).all() and (V[0] == 4).all() and c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK


def test_append_reports_every_sequence_that_it_refuses():
    """Sequences whose rows or length make no sense are reported by append too, also where no row of the call is theirs;
    nothing of them is written, and the others are."""
    kvh, dh, page = 2, 64, 16
    c = Paged([20, 40, 3], [1, 1, 1], kvh, kvh, dh, page, "bf16", seed=19)
    k, v = c.rows(kvh), c.rows(kvh)
    c.cache.append(None, k, v, c.gtable, c.glens, None)
    pool = c.cache.pool.clone()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for start, lens, written in ((i32(0, 5, -3, 2 ** 30), c.glens, ()),        # starts beyond the rows, and falling
                                 (i32(0, 3, 3, 3), i32(2, 40, 3), ()),         # fewer tokens than new ones
                                 (i32(2, 1, 2, 3), c.glens, (1, 2)),           # a sequence that begins behind its end
                                 (i32(0, 1, 1, 2), i32(20, 10 ** 9, 3), (0, 2)),   # no new tokens, but a length past the table
                                 (i32(0, 1, 1, 2), i32(20, -1, 3), (0, 2))):
        c.cache.pool.zero_()
        c.cache.append(None, k, v, c.gtable, lens, start)
        assert c.cache.last_device_error()[0] == sp.ERR_DEVICE_CHECK, start.tolist()
        got = c.cache.pool.view(c.pages, -1).ne(0).any(1).cpu()
        assert got.sum() == len(written) and all(got[c.table[b, (c.lens[b] - 1) // page]] for b in written), start.tolist()
    c.cache.pool.zero_()
    c.cache.append(None, k, v, c.gtable, c.glens, i32(0, 1, 2, 3))
    assert torch.equal(c.cache.pool, pool) and c.cache.last_device_error() == (sp.OK, 0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("unit", [1.0, 0.25, 2.0 ** -10, 3.0])
def test_append_codes_at_and_beside_halves(dtype, unit):
    """Quotients that are halves (ties to even) and the numbers next to them: the codes are those of the exact division."""
    base = np.concatenate([[0.0, 15.0], np.arange(15) + 0.5, np.arange(15) + 0.25])[:32] * unit
    rows = []
    for shift in (0, 1, -1):
        x = torch.tensor(base, dtype=torch.float64).to(DT[dtype])
        x[2:] = (x[2:].view(torch.int16) + shift).view(DT[dtype])       # the next number up or down
        rows.append(torch.cat([x, x.flip(0)]))
    v = torch.stack(rows).view(3, 1, 64).cuda()
    c = Paged([1, 1, 1], [1, 1, 1], 1, 1, 64, 16, dtype, seed=60)
    c.cache.append(None, v, v, c.gtable, c.glens, None)
    codes = OB.read_pool(c.cache.pool.cpu().numpy(), 16, 1, 64)
    for name in "KV":
        for got, want in zip(codes[name], OB.quantise(f64(v).astype(np.float32))):
            assert np.array_equal(got[c.table[:3, 0], 0], want)


def test_append_then_attend_replays_in_a_graph():
    """A captured decode step: lengths grow on the device, every replay appends the next token and attends to it."""
    nh, kvh, dh, page, steps = 8, 2, 128, 16, 20
    c = Paged([16 + steps, 5 + steps], [1, 1], nh, kvh, dh, page, "bf16", seed=14, rope=(10000.0 ** (-np.arange(64) / 64), False, 1.0))
    c.fill(nan_behind=False)
    q, k, v = c.rows(nh), c.rows(kvh), c.rows(kvh)
    qo, out = torch.empty_like(q), torch.empty_like(q)
    lens = torch.tensor([16, 5], dtype=torch.int32, device="cuda")

    def step():
        lens.add_(1)
        c.cache.append(q, k, v, c.gtable, lens, None, qo)
        c.cache.attend(qo, c.gtable, lens, None, out)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(steps - 1):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = OB.read_pool(c.cache.pool.cpu().numpy(), page, kvh, dh)
        c.K, c.V, c.lens = got["K"], got["V"], lens.tolist()
        c.check_attend(qo, out)
    assert lens.tolist() == c.lens == [16 + steps, 5 + steps] and c.cache.last_device_error() == (sp.OK, 0)


# ------------------------------------------------------------------------------- the whole block
def test_block_around_the_sparse_ffn():
    """norm -> q/k/v -> append -> attend -> 8-bit rows -> output product -> norm -> sparse FFN, three decode
    steps of a batch; every stage is held to the oracle on the stage's own input."""
    import workload as wl
    cfg = wl.CONFIGS[0]
    d, B, nh, kvh, dh, page = cfg.d, 5, 8, 4, 128, 16
    h = wl.host_layer(cfg, 0)
    t = lambda a: wl.to_torch(a, cfg, "cuda:0")  # noqa: E731
    ffn = sp.Layer(t(h.W1), t(h.b1), t(h.W2T), t(h.b2), t(h.Wp1), t(h.bp1), t(h.Wp2), t(h.bp2), max_batch=8)
    dtype, name = (torch.bfloat16, "bf16") if cfg.bf16 else (torch.float16, "f16")
    gen = torch.Generator(device="cuda").manual_seed(21)
    w = lambda n, k: (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(dtype)  # noqa: E731

    def product(W):
        q, s = torch.empty(W.shape, dtype=torch.int8, device="cuda"), torch.empty(W.shape[0], device="cuda")
        sp.quantize_rows(W, q, s)
        return sp.Linear8(q, s, None, max_tokens=8, dtype=dtype)

    qkv, proj = product(w((nh + 2 * kvh) * dh, d)), product(w(d, nh * dh))
    freqs, _ = sp.rope_frequencies(dh)
    steps, lens0 = 3, [0, 15, 16, 3, 40]
    c = Paged([n + steps for n in lens0], [1] * B, nh, kvh, dh, page, name, seed=22, rope=(freqs, False, 1.0))
    c.fill(nan_behind=False)
    lens = dev(np.array(lens0, np.int32))
    g1, g2 = ((1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dtype) for _ in range(2))
    x = torch.randn(B, d, generator=gen, device="cuda").to(dtype)
    y = torch.zeros(B, d, device="cuda")
    e = lambda *s, k=dtype: torch.empty(*s, dtype=k, device="cuda")  # noqa: E731
    q8, s8, x1, x2 = e(B, d, k=torch.int8), e(B, k=torch.float32), e(B, d), e(B, d)
    joint, qo, att, o = e(B, (nh + 2 * kvh) * dh), e(B, nh, dh), e(B, nh, dh), e(B, d)
    a8, as8, f8, fs8 = e(B, nh * dh, k=torch.int8), e(B, k=torch.float32), e(B, d, k=torch.int8), e(B, k=torch.float32)
    idx, cnt = e(cfg.n, k=torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
    W64 = {n: h.f64(n) for n in ("W1", "b1", "W2T", "b2")}
    for _ in range(steps):
        lens += 1
        y_in, x_in = y.clone(), x.clone()
        sp.norm_quant(x, y, g1, x1, q8, s8)
        qkv.forward(q8, s8, joint)
        hq, hk = nh * dh, (nh + kvh) * dh
        c.cache.append(joint[:, :hq], joint[:, hq:hk], joint[:, hk:], c.gtable, lens, None, qo)
        c.cache.attend(qo, c.gtable, lens, None, att)
        sp.quantize_rows(att.view(B, -1), a8, as8)
        proj.forward(a8, as8, o)
        sp.norm_quant(x1, o, g2, x2, f8, fs8)
        xn = (f8.float() * fs8[:, None]).to(dtype)
        ffn.step(xn, idx, cnt, y)
        torch.cuda.synchronize()
        check_norm(x_in, y_in, g1, 1e-6, x1, q8, s8, name)
        check_mm8(joint, q8, qkv._keep[0], s8, qkv._keep[1], None, name)
        got = OB.read_pool(c.cache.pool.cpu().numpy(), page, kvh, dh)
        c.K, c.V, c.lens = got["K"], got["V"], lens.tolist()
        c.check_attend(qo, att)
        check_mm8(o, a8, proj._keep[0], as8, proj._keep[1], None, name)
        check_norm(x1, o, g2, 1e-6, x2, f8, fs8, name)
        k = int(cnt.item())
        want = O.sparse_ffn(W64["W1"], W64["b1"], W64["W2T"], W64["b2"], f64(xn), idx[:k].cpu().numpy())
        assert np.linalg.norm(f64(y) - want) <= 1e-3 * np.linalg.norm(want)
        x = x2.clone()
    assert c.cache.last_device_error() == (sp.OK, 0) and qkv.last_device_error() == (sp.OK, 0)
