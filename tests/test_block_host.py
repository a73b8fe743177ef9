"""The dense half of a batched decode block on CPU: refusals at the C entry points (host
checks, before anything is enqueued), workspace and pool sizes, rotary frequencies, and
the oracle's own pins."""
import ctypes
import math
import subprocess

import numpy as np
import pytest

import activation_sparse_ffn_predictor_b200 as sp
import oracle.block as OB
from activation_sparse_ffn_predictor_b200 import build

F = 1 << 40     # an address that host checks never dereference
BAD = sp.ERR_INVALID_ARG


def test_norm_refusals():
    f = sp.library().spffn_norm_quant
    #          T  d   dt  x  ldx y  ldy f32 g  eps   xo ldo q  ldq scale stream
    ok = dict(T=0, d=64, dt=0, x=F, ldx=64, y=F, ldy=64, f32=1, g=F, eps=1e-6, xo=F + 4096, ldo=64, q=F, ldq=64, s=F, st=None)
    assert f(*ok.values()) == sp.OK                       # no rows: nothing to do
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(dt=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf),
                dict(eps=math.nan)):
        assert f(*{**ok, **bad}.values()) == BAD, bad
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(ldx=63), dict(ldy=63), dict(ldo=63), dict(ldq=63),
                dict(x=F + 1), dict(y=F + 2), dict(s=F + 2), dict(g=F + 1), dict(xo=F, ldo=128), dict(xo=F + 1),
                dict(xo=F, x=F + 64)):
        assert f(*{**ok, "T": 3, **bad}.values()) == BAD, bad    # the last: y is fp32, x_out may not be y


def test_quantize_rows_refusals():
    f = sp.library().spffn_quantize_rows
    ok = dict(T=0, d=64, dt=0, x=F, ldx=64, f32=0, q=F, ldq=64, s=F, st=None)
    assert f(*ok.values()) == sp.OK
    for bad in (dict(T=-1), dict(d=0), dict(d=131073), dict(dt=7), dict(T=1, x=None), dict(T=1, q=None), dict(T=1, s=None),
                dict(T=1, ldx=63), dict(T=1, ldq=63), dict(T=1, x=F + 2, f32=1), dict(T=1, s=F + 1)):
        assert f(*{**ok, **bad}.values()) == BAD, bad


def mm8(K=256, N=100, max_tokens=8, dtype=0, flags=0):
    return sp.Mm8Config(K, N, max_tokens, dtype, flags)


def test_mm8_refusals():
    lib = sp.library()
    size = lambda c: lib.spffn_mm8_workspace_bytes(ctypes.byref(c))  # noqa: E731
    need = size(mm8())
    assert need > 0
    for bad in (mm8(K=0), mm8(K=24), mm8(K=131088), mm8(N=0), mm8(N=262145), mm8(max_tokens=0), mm8(max_tokens=1 << 21),
                mm8(dtype=2), mm8(flags=1)):
        assert size(bad) == 0
    ctx = ctypes.c_void_p()
    create = lambda c, w, ws, n: lib.spffn_mm8_create(ctypes.byref(c), ctypes.byref(w), ws, n, ctypes.byref(ctx))  # noqa: E731
    w = sp.Mm8Weights(F, F, F)
    assert create(mm8(K=24), w, F, need) == BAD
    for bad in (sp.Mm8Weights(None, F, F), sp.Mm8Weights(F, None, F), sp.Mm8Weights(F + 8, F, F), sp.Mm8Weights(F, F + 2, F),
                sp.Mm8Weights(F, F, F + 1)):
        assert create(mm8(), bad, F, need) == BAD
    assert create(mm8(), w, None, need) == sp.ERR_WORKSPACE
    assert create(mm8(), w, F + 16, need) == sp.ERR_WORKSPACE
    assert create(mm8(), w, F, need - 1) == sp.ERR_WORKSPACE
    assert create(mm8(), w, F, need) == sp.OK
    f = lib.spffn_mm8_forward
    ok = dict(ctx=ctx, A=F, lda=256, s=F, T=0, y=F, ldy=100, st=None)
    assert f(*ok.values()) == sp.OK
    for bad in (dict(ctx=None), dict(T=-1), dict(T=9), dict(A=None), dict(s=None), dict(y=None), dict(lda=240), dict(lda=264),
                dict(ldy=99), dict(A=F + 8), dict(s=F + 2), dict(y=F + 1)):
        assert f(*{**ok, "T": 3, **bad}.values()) == BAD, bad
    assert lib.spffn_mm8_last_device_error(None, None, None) == BAD
    assert lib.spffn_mm8_destroy(ctx) == sp.OK and lib.spffn_mm8_destroy(None) == sp.OK


def kv4(pages=4, page=16, nh=8, kvh=2, dh=64, seqs=3, tokens=9, dtype=1, rd=64, inter=0, amp=1.0, flags=0):
    return sp.Kv4Config(pages, page, nh, kvh, dh, seqs, tokens, dtype, rd, inter, flags, amp)


def test_kv4_refusals():
    lib = sp.library()
    size = lambda c: lib.spffn_kv4_pool_bytes(ctypes.byref(c))  # noqa: E731
    assert size(kv4()) == 4 * 2 * 16 * (64 + 64) * 5 // 8      # 5 bits a value with steps and zeros
    for bad in (kv4(pages=0), kv4(pages=(1 << 24) + 1), kv4(page=8), kv4(page=48), kv4(nh=0), kv4(nh=7), kv4(nh=1025, kvh=1025),
                kv4(nh=130, kvh=2), kv4(dh=96), kv4(seqs=0), kv4(seqs=4097), kv4(tokens=0), kv4(tokens=65537), kv4(dtype=2),
                kv4(rd=-2), kv4(rd=66), kv4(rd=3), kv4(amp=math.nan), kv4(flags=1)):
        assert size(bad) == 0 and lib.spffn_kv4_workspace_bytes(ctypes.byref(bad)) == 0
    big = kv4(pages=1 << 20, page=64, kvh=8, nh=64, dh=128)
    assert size(big) == (1 << 20) * 64 * 8 * 160               # past 32 bits
    need, pool = lib.spffn_kv4_workspace_bytes(ctypes.byref(kv4())), size(kv4())
    ctx = ctypes.c_void_p()

    def create(c=kv4(), at=F, n=pool, freqs=F, ws=F, m=need):
        return lib.spffn_kv4_create(ctypes.byref(c), at, n, freqs, ws, m, ctypes.byref(ctx))

    for bad in (dict(c=kv4(page=8)), dict(at=None), dict(at=F + 16), dict(n=pool - 1), dict(freqs=None), dict(freqs=F + 4)):
        assert create(**bad) == BAD, bad
    for bad in (dict(ws=None), dict(ws=F + 16), dict(m=need - 1)):
        assert create(**bad) == sp.ERR_WORKSPACE, bad
    assert create() == sp.OK
    f = lib.spffn_kv4_append
    ok = dict(ctx=ctx, q=F, ldq=512, k=F, ldk=128, v=F, ldv=128, T=5, table=F, ldt=4, width=4, lens=F, start=F, B=2, qo=F,
              ldqo=512, st=None)
    for none in (dict(T=0), dict(B=0)):
        assert f(*{**ok, **none}.values()) == sp.OK
    for bad in (dict(ctx=None), dict(T=-1), dict(T=10), dict(B=-1), dict(B=4), dict(q=None), dict(qo=None), dict(k=None),
                dict(v=None), dict(ldq=511), dict(ldk=127), dict(ldv=127), dict(ldqo=511), dict(ldqo=1024), dict(table=None),
                dict(ldt=3), dict(width=0), dict(lens=None), dict(q=F + 1), dict(k=F + 1), dict(v=F + 1), dict(table=F + 2),
                dict(lens=F + 2), dict(start=F + 2), dict(start=None, T=1)):
        assert f(*{**ok, **bad}.values()) == BAD, bad
    f = lib.spffn_kv4_attend
    ok = dict(ctx=ctx, q=F, ldq=512, T=5, table=F, ldt=4, width=4, lens=F, start=F, B=2, scale=0.125, out=F + 65536, ldo=512, st=None)
    for none in (dict(T=0), dict(B=0)):
        assert f(*{**ok, **none}.values()) == sp.OK
    for bad in (dict(ctx=None), dict(T=10), dict(B=4), dict(q=None), dict(out=None), dict(out=F), dict(ldq=511), dict(ldo=511),
                dict(scale=math.nan), dict(scale=math.inf), dict(q=F + 1), dict(out=F + 1), dict(width=-1)):
        assert f(*{**ok, **bad}.values()) == BAD, bad
    f = lib.spffn_kv4_read
    assert f(ctx, F, 0, F, F, None) == sp.OK
    for bad in ((None, F, 1, F, F + 4096, None), (ctx, None, 1, F, F + 4096, None), (ctx, F, -1, F, F + 4096, None), (ctx, F, 1, F, F, None),
                (ctx, F, 1, F + 8, F + 4096, None), (ctx, F, 1, F, None, None), (ctx, F, 1 << 30, F, F + 4096, None)):
        if bad[2] != 1 << 30:
            assert f(*bad) == BAD, bad
    assert lib.spffn_kv4_last_device_error(None, None, None) == BAD
    assert lib.spffn_kv4_destroy(ctx) == sp.OK and lib.spffn_kv4_destroy(None) == sp.OK


JOIN = r"""
#include <cstdio>
#include <cstdint>
#include "spffn_kv4.cuh"
using namespace spffn::kv4;
int main() {
    // entries as a call of 1776 shares of 8 rows leaves them, and any bits, read in calls of every shape
    unsigned long long r = 1, bad = 0, in = 0, lost = 0;
    for (int many = 1; many <= 148 * 16; many = many * 5 / 4 + 1)
        for (int R : {8, 16, 32})
            for (int i = 0; i < 20000; ++i) {
                r = r * 6364136223846793005ull + 1442695040888963407ull;
                const uint32_t a = (uint32_t)(r >> 32);
                r = r * 6364136223846793005ull + 1442695040888963407ull;
                const uint32_t b = (uint32_t)(r >> 32);
                const uint2 m = i % 2 ? uint2{a, b >> (b & 31)} : pack_cuts(Cuts{a % 1776, b % 200, (a >> 16) % 8});
                const Cuts c = unpack_cuts(m);
                const bool ok = cuts_in(c, many, R);
                // the parts are [2 many][R rows]: share s has places 2 s and 2 s + 1
                const bool inside = (unsigned long long)c.first + c.more < (unsigned long long)many && c.in < (uint32_t)R;
                bad += ok && !inside;
                lost += inside && !ok;
                in += ok;
            }
    for (uint32_t first : {0u, 1u, 1775u, 0xffffffu})
        for (uint32_t place : {0u, 7u, 31u, 255u}) {
            const Cuts c = unpack_cuts(pack_cuts(Cuts{first, 9u, place}));
            bad += c.first != first || c.more != 9u || c.in != place;
        }
    std::printf("%llu %llu %d\n", bad, lost, in > 1000);
}
"""


def test_join_stays_inside_the_workspace(tmp_path):
    """Whatever an entry holds, the join follows it only to parts that the call's workspace has."""
    src, exe = tmp_path / "join.cu", tmp_path / "join"
    src.write_text(JOIN)
    subprocess.check_call([build.NVCC, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-o", str(exe), str(src)])
    assert subprocess.check_output([str(exe)]).split() == [b"0", b"0", b"1"]


def test_binding_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    x, q, s = torch.zeros(2, 64, dtype=torch.float16), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        sp.Linear8(torch.zeros(8, 16, dtype=torch.int8), torch.zeros(8))
    for a in (dict(x=x, y=None, g=None, x_out=None, q=q, scale=s), dict(x=x, y=x, g=x[0], x_out=x, q=q, scale=s)):
        with pytest.raises(TypeError):     # host memory never reaches a kernel
            sp.norm_quant(**a)
    with pytest.raises(TypeError):
        sp.quantize_rows(x, q, s)
    for bad in (dict(q=q[:, :63]), dict(q=q.float()), dict(scale=s[:1]), dict(g=s), dict(y=q), dict(x_out=q)):
        a = dict(x=x, y=None, g=None, x_out=None, q=q, scale=s)
        with pytest.raises((ValueError, TypeError)):
            sp.norm_quant(**{**a, **bad})


def test_rope_frequencies():
    n = 32
    plain, amp = sp.rope_frequencies(2 * n, 10000.0)
    want = 10000.0 ** (-np.arange(n) / n)
    assert np.allclose(plain, want, rtol=1e-14, atol=0) and amp == 1.0
    assert np.allclose(sp.rope_frequencies(2 * n, 10000.0, "linear", 4.0)[0], want / 4, rtol=1e-14, atol=0)
    ntk = sp.rope_frequencies(2 * n, 10000.0, "ntk", 4.0)[0]
    assert math.isclose(ntk[0], 1.0) and math.isclose(ntk[-1], want[-1] / 4, rel_tol=1e-12)   # the slowest pair is interpolated
    parts, amp = sp.rope_frequencies(2 * n, 10000.0, "parts", 8.0, 4096.0)
    turns = 4096 * want / (2 * math.pi)
    assert math.isclose(amp, 0.1 * math.log(8.0) + 1, rel_tol=1e-6)
    assert np.allclose(parts[turns >= 32], want[turns >= 32], rtol=1e-14, atol=0)
    assert np.allclose(parts[turns <= 1], want[turns <= 1] / 8, rtol=1e-14, atol=0)
    between = (turns > 1) & (turns < 32)
    assert between.any() and np.all(parts[between] < want[between]) and np.all(parts[between] > want[between] / 8)
    for bad in (dict(dim=0), dict(dim=3), dict(dim=8, base=0.0), dict(dim=8, scaling="linear", factor=0.5),
                dict(dim=2, scaling="ntk", factor=2.0), dict(dim=8, scaling="parts", factor=2.0)):
        with pytest.raises(sp.SpffnError):
            sp.rope_frequencies(**bad)
    with pytest.raises(ValueError):
        sp.rope_frequencies(8, scaling="other")


class Recorder:
    """Stands in for torch and the library where a second device would be needed: what is called, on which device."""

    def __init__(self, current):
        self.current, self.calls = current, []
        self.cuda = self

    def is_current_stream_capturing(self):
        return False

    def current_stream(self, device):
        return self

    def synchronize(self):
        pass

    def device(self, index):
        outer = self

        class Guard:
            def __enter__(self):
                self.before, outer.current = outer.current, index

            def __exit__(self, *_):
                outer.current = self.before
        return Guard()

    def __getattr__(self, name):
        if not name.startswith("spffn_"):
            raise AttributeError(name)
        return lambda *a: self.calls.append((name, self.current, a[-1])) or sp.OK


@pytest.mark.parametrize("cls", [sp.Linear8, sp.KvCache4])
def test_device_errors_are_read_on_the_contexts_own_device(cls, monkeypatch):
    """The error word is read after what was enqueued on the context's device, whichever device is current."""
    rec = Recorder(0)
    for name, value in (("_T", rec), ("_lib", rec), ("_device_now", lambda: rec.current), ("_stream_now", lambda d: 100 + d)):
        monkeypatch.setattr(sp, name, value)
    obj = cls.__new__(cls)
    obj.ctx, obj.device = None, 1
    assert obj.last_device_error() == (sp.OK, 0)
    assert obj.last_device_error(stream=7) == (sp.OK, 0)
    (_, at, stream), (_, at2, stream2) = rec.calls
    assert (at, stream, at2, stream2) == (1, 101, 1, 7) and rec.current == 0


def test_linear8_refuses_a_workspace_of_another_device(monkeypatch):
    torch = pytest.importorskip("torch")

    class Fake:
        def __init__(self, device, dtype, *shape):
            self.where, self.dtype, self.shape, self.device, self.is_cuda = device, dtype, shape, "cuda:%d" % device, True

        def get_device(self):
            return self.where

        def stride(self):
            return self.shape[1:] + (1,)

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return F

        def numel(self):
            return self.shape[0]

    rec = Recorder(0)
    rec.float16, rec.bfloat16, rec.int8, rec.float32 = torch.float16, torch.bfloat16, torch.int8, torch.float32
    monkeypatch.setattr(sp, "_T", rec)
    made = lambda where: sp.Linear8(Fake(1, torch.int8, 8, 64), Fake(1, torch.float32, 8), workspace=Fake(where, torch.uint8, 1 << 30))  # noqa: E731
    assert made(1).device == 1
    with pytest.raises(ValueError):
        made(0)


def test_read_refuses_what_no_grid_holds():
    lib, ctx = sp.library(), ctypes.c_void_p()
    c = kv4(pages=1 << 24, page=256, nh=1024, kvh=1024, dh=256, rd=0)
    assert lib.spffn_kv4_create(ctypes.byref(c), F, lib.spffn_kv4_pool_bytes(ctypes.byref(c)), None, F,
                                lib.spffn_kv4_workspace_bytes(ctypes.byref(c)), ctypes.byref(ctx)) == sp.OK
    assert lib.spffn_kv4_read(ctx, F, 1 << 20, F, F + 4096, None) == BAD       # 2^34 blocks of 16 tokens
    lib.spffn_kv4_destroy(ctx)


def test_device_errors_are_refused_on_another_device():
    """Here no device is current at all: nothing is enqueued."""
    lib, ctx, code = sp.library(), ctypes.c_void_p(), ctypes.c_uint32(0)
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a device is current")
    c, w = mm8(), sp.Mm8Weights(F, F, F)
    assert lib.spffn_mm8_create(ctypes.byref(c), ctypes.byref(w), F, lib.spffn_mm8_workspace_bytes(ctypes.byref(c)), ctypes.byref(ctx)) == sp.OK
    assert lib.spffn_mm8_last_device_error(ctx, ctypes.byref(code), None) == BAD
    lib.spffn_mm8_destroy(ctx)
    c = kv4()
    assert lib.spffn_kv4_create(ctypes.byref(c), F, lib.spffn_kv4_pool_bytes(ctypes.byref(c)), F, F,
                                lib.spffn_kv4_workspace_bytes(ctypes.byref(c)), ctypes.byref(ctx)) == sp.OK
    assert lib.spffn_kv4_last_device_error(ctx, ctypes.byref(code), None) == BAD
    lib.spffn_kv4_destroy(ctx)


def test_attend_says_that_it_wants_an_output():
    torch = pytest.importorskip("torch")
    c = sp.KvCache4.__new__(sp.KvCache4)
    c.ctx, c.nh, c.kvh, c.dh, c.dtype = None, 2, 1, 64, torch.float16
    q, i = torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError, match="out"):
        c.attend(q, i, i[0])
    with pytest.raises(TypeError, match="v"):
        c.append(None, q[:, :1], None, i, i[0])


def test_rope_amplitude_keeps_its_bits():
    """The config takes the amplitude as a double, and codes are decided by it: it is not rounded on its way there."""
    for factor in (1.5, 8.0, 40.0):
        assert math.isclose(sp.rope_frequencies(64, 10000.0, "parts", factor, 4096.0)[1], 0.1 * math.log(factor) + 1, rel_tol=1e-15)


def test_oracle_pool_round_trip():
    r = np.random.default_rng(3)
    for dh, kvh, page in ((64, 3, 16), (128, 1, 32), (256, 2, 16)):
        K, V = (OB.quantise(r.normal(size=(2, page, kvh, dh)).astype(np.float32)) for _ in range(2))
        got = OB.read_pool(OB.write_pool(K, V, page, kvh, dh), page, kvh, dh)
        for name, want in (("K", K), ("V", V)):
            for a, b in zip(got[name], want):
                assert np.array_equal(a, b)


def test_oracle_quantise_is_within_half_a_step():
    r = np.random.default_rng(4)
    x = r.normal(size=(50, 64)) * np.exp(r.normal(size=(50, 1)) * 3)
    c, s, z = OB.quantise(x.astype(np.float32))
    step = np.repeat(s.astype(np.float64), 32, -1)
    lo = np.abs(np.repeat(z.astype(np.float64), 32, -1))
    # half a step, plus what the fp16 roundings of zero and step move the ends of the range
    assert np.all(np.abs(OB.values(c, s, z) - x) <= step / 2 + 2.0 ** -11 * (lo + 15 * step) + 2.0 ** -24)


def test_oracle_attend_against_a_loop():
    r = np.random.default_rng(5)
    q, K, V = r.normal(size=(3, 8)), r.normal(size=(5, 8)), r.normal(size=(5, 8))
    vis = np.array([[1, 1, 0, 0, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1]], bool)
    o, _ = OB.attend(q, K, V, vis, 0.3)
    for i in range(3):
        ks = [j for j in range(5) if vis[i, j]]
        e = [math.exp(0.3 * float(q[i] @ K[j])) for j in ks]
        want = sum(w * V[j] for w, j in zip(e, ks)) / sum(e) if ks else np.zeros(8)
        assert np.allclose(o[i], want, rtol=1e-12, atol=1e-14)


def test_oracle_rotation_keeps_pair_lengths_and_is_relative():
    r = np.random.default_rng(6)
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        a, b = r.normal(size=(1, 1, 64)), r.normal(size=(1, 1, 64))
        turn = lambda x, p: OB.rotate(x, [p], f, inter)  # noqa: E731
        assert np.isclose(np.linalg.norm(turn(a, 9)), np.linalg.norm(a))
        assert np.allclose(turn(a, 7)[..., 32:], a[..., 32:])
        # scores depend on the distance of the positions alone
        assert np.isclose((turn(a, 12) * turn(b, 5)).sum(), (turn(a, 107) * turn(b, 100)).sum())
