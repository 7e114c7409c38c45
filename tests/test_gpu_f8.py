"""8-bit matrices on the GPU: quantize bit for bit against tests/f8_ref.py,
products against 64 bits and exactly where every sum is a whole number, and a
layer's forward and backward pass into the AdamW step."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import zero_sharded_mixed_zero1_amd as z
from tests import f8_ref as ref
from tests import state8_ref as ref8
from tests.gpu_util import assert_f32_equal, torch_cuda, ws_tensor
from tests.test_gpu_state8 import Buf, bf16_bits, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


def up(n, a):
    return -(-n // a) * a


class Mat:
    """An 8-bit matrix between guards; `wide` bytes of stride more than the least, `tall` more of the scales."""

    def __init__(self, env, rows, cols, block=1, e5m2=False, wide=0, more=0, fill=0xA7):
        torch, dev = env
        self.rows, self.cols, self.block, self.e5m2 = rows, cols, block, e5m2
        self.ld, self.lds = up(cols, 128) + wide, up(ref.ceil(cols), 4) + more
        self.srows = -(-rows // block)
        self.codes, self.scales = Buf(torch, dev, rows * self.ld, fill=fill), Buf(torch, dev, self.srows * self.lds, fill=fill)
        self.m = z.f8_matrix(rows, cols, self.codes.view, self.scales.view, block_rows=block, flags=z.E5M2 if e5m2 else 0,
                             ld=self.ld if wide else 0, ld_scales=self.lds if more else 0)

    def put(self, codes, scales):
        c = np.full((self.rows, self.ld), 0xA7, np.uint8)
        c[:, :up(self.cols, 128)] = 0
        c[:, :self.cols] = codes
        s = np.full((self.srows, self.lds), 0xA7, np.uint8)
        s[:, :ref.ceil(self.cols)] = scales
        self.codes.put(c.reshape(-1))
        self.scales.put(s.reshape(-1))
        return self

    def get(self):
        return self.codes.get().reshape(self.rows, self.ld), self.scales.get().reshape(self.srows, self.lds)

    def check(self, x, what):
        """Holds the quantized x, zeros up to whole blocks, and nothing else."""
        codes, scales = ref.quantize(x, self.block, self.e5m2)
        c, s = self.get()
        got, nan = c[:, :self.cols], np.isnan(x)
        want = ref.TABLE[self.e5m2][codes]
        want = np.where(np.isinf(x), np.copysign(np.inf, x) if self.e5m2 else np.nan, np.where(nan, np.nan, want))
        assert np.array_equal(s[:, :ref.ceil(self.cols)], scales), f"scales {what}"
        v = ref.TABLE[self.e5m2][got]
        assert np.array_equal(np.isnan(v), np.isnan(want)), f"NaN {what}"
        keep = np.isfinite(x)
        assert np.array_equal(got[keep], codes[keep]), f"codes {what}: {(got[keep] != codes[keep]).sum()} differ"
        assert np.array_equal(v[np.isinf(want)], want[np.isinf(want)])
        assert (c[:, self.cols:up(self.cols, 128)] == 0).all(), f"padding {what}"
        assert (c[:, up(self.cols, 128):] == 0xA7).all() and (s[:, ref.ceil(self.cols):] == 0xA7).all(), f"written beside {what}"
        assert self.codes.guards_hold() and self.scales.guards_hold(), f"guards {what}"


def source(env, rows, cols, seed, f32, pad=0, skew=0, spread=2.0):
    """Values [rows, cols] in a buffer with `pad` more elements a row, `skew` elements off its alignment."""
    torch, dev = env
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1))) * np.exp(spread * rng.standard_normal((rows, cols)))).astype(np.float32)
    if not f32:
        x = widen(bf16_bits(x))
    return x, device_source(env, x, f32, pad, skew)


def device_source(env, x, f32, pad=0, skew=0):
    torch, dev = env
    rows, cols = x.shape
    full = np.full((rows, cols + pad), 3e38, np.float32)
    full[:, :cols] = x
    e = 4 if f32 else 2
    buf = Buf(torch, dev, full.size * e, skew=skew * e)
    buf.put(full.reshape(-1) if f32 else bf16_bits(full.reshape(-1)))
    return buf


SHAPES = [(1, 1), (1, 128), (128, 1), (7, 129), (127, 127), (128, 128), (129, 300), (200, 8), (1, 5000), (5000, 1), (513, 1023)]


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("block,block_t,e5,e5t", [(1, 1, False, False), (128, 128, False, True), (1, 128, True, False), (128, 1, True, True)])
def test_quantize(env, rows, cols, f32, block, block_t, e5, e5t):
    x, src = source(env, rows, cols, rows * 7 + cols, f32)
    q, qt = Mat(env, rows, cols, block, e5), Mat(env, cols, rows, block_t, e5t)
    z.f8_quantize(src.view, rows, cols, q=q.m, qt=qt.m, flags=z.F32 if f32 else 0)
    q.check(x, "along")
    qt.check(np.ascontiguousarray(x.T), "across")
    # one of the two alone
    q1, q2 = Mat(env, rows, cols, block, e5), Mat(env, cols, rows, block_t, e5t)
    z.f8_quantize(src.view, rows, cols, q=q1.m, flags=z.F32 if f32 else 0)
    z.f8_quantize(src.view, rows, cols, qt=q2.m, flags=z.F32 if f32 else 0)
    q1.check(x, "along alone")
    q2.check(np.ascontiguousarray(x.T), "across alone")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad,skew", [(1, 0), (23, 3), (8, 1)])
def test_quantize_strides_and_alignment(env, f32, pad, skew):
    rows, cols = 261, 390
    x, src = source(env, rows, cols, 5, f32, pad, skew)
    q, qt = Mat(env, rows, cols, 1, wide=48, more=8), Mat(env, cols, rows, 128, wide=16, more=4)
    z.f8_quantize(src.view, rows, cols, q=q.m, qt=qt.m, ld=cols + pad, flags=z.F32 if f32 else 0)
    q.check(x, "along")
    qt.check(np.ascontiguousarray(x.T), "across")
    assert src.guards_hold()


def test_quantize_special_values(env):
    """NaN and infinities in one block leave the other values' scale alone; blocks of zeros, of the smallest and the
    largest values, and values at the borders of the formats."""
    rows, cols = 256, 384
    rng = np.random.default_rng(3)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x[0, 0], x[1, 1], x[2, 2] = np.nan, np.inf, -np.inf
    x[5, :128] = np.nan
    x[6, :128] = np.inf
    x[7, :128] = 0.0
    x[8, :128] = -0.0
    x[9, :128] = np.float32(2.0 ** -149) * np.arange(128)
    x[10, :128] = np.float32(3.4e38) * rng.uniform(-1, 1, 128).astype(np.float32)
    x[11, 128:256] = 2.0 ** -126
    x[12, 128:256] = np.float32(448) * (1 + np.arange(128) * 2.0 ** -23).astype(np.float32)
    x[13, 128:256] = np.float32(448)
    x[14, 128:256] = np.float32(57344)
    x[15, 128:256] = [464 if k % 2 else 17 for k in range(128)]      # ties
    x[16, 128:256] = 448 * 2.0 ** (-(np.arange(128) % 40).astype(np.float64))
    for f32 in (True, False):
        y = x if f32 else widen(bf16_bits(x))
        src = device_source(env, y, f32)
        for block, e5 in ((1, False), (1, True), (128, False), (128, True)):
            q, qt = Mat(env, rows, cols, block, e5), Mat(env, cols, rows, block, e5)
            z.f8_quantize(src.view, rows, cols, q=q.m, qt=qt.m, flags=z.F32 if f32 else 0)
            q.check(y, "along")
            qt.check(np.ascontiguousarray(y.T), "across")


def test_empty_matrices(env):
    torch, dev = env
    src = torch.ones(10, device=dev)
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        z.f8_quantize(src, rows, cols, q=z.f8_matrix(rows, cols, None, None), qt=z.f8_matrix(cols, rows, None, None), flags=z.F32)
    b = Mat(env, 7, 300).put(np.ones((7, 300), np.uint8), np.full((7, 3), 127, np.uint8))
    d = torch.full((3, 7), 5.0, device=dev)
    z.f8_product(z.f8_matrix(0, 300, None, None), b.m, d, flags=z.F32)
    z.f8_product(b.m, z.f8_matrix(0, 300, None, None), d, flags=z.F32)
    torch.cuda.synchronize()
    assert (d == 5.0).all()
    # no columns: sums of nothing
    z.f8_product(z.f8_matrix(3, 0, None, None), z.f8_matrix(7, 0, None, None), d, flags=z.F32)
    assert (d == 0.0).all()


# ------------------------------------------------------------------ product
def product(env, a, b, f32, ld_more=0, ws=None, stream=None, skew=0):
    """d between guards, the elements beside its columns checked; as fp32 values."""
    torch, dev = env
    e, n = (4 if f32 else 2), b.rows + ld_more
    d = Buf(torch, dev, a.rows * n * e, skew=skew)
    flags = z.F32 if f32 else 0
    need = z.f8_product_workspace_bytes(a.m, b.m, flags)
    if ws is None:
        ws = ws_tensor(torch, need, dev)
    z.f8_product(a.m, b.m, d.view, ldd=n if ld_more else 0, flags=flags, ws=ws, stream=stream)
    got = d.get(np.uint32 if f32 else np.uint16).reshape(a.rows, n)
    assert d.guards_hold()
    assert (got[:, b.rows:] == (0xA7A7A7A7 if f32 else 0xA7A7)).all(), "written beside d's columns"
    got = np.ascontiguousarray(got[:, :b.rows])
    return got.view(np.float32) if f32 else widen(got)


def whole_numbers(env, rows, cols, seed, block, e5m2, wide=0, more=0):
    """Whole numbers from -2 to 2 (exact in every sum below 2^22 columns) with scales of 1, 2 and 4."""
    rng = np.random.default_rng(seed)
    v = rng.integers(-2, 3, (rows, cols)).astype(np.float64)
    t = ref.TABLE[e5m2]
    codes = np.array([int(np.flatnonzero((t == k) & (np.signbit(t) == (k < 0)))[0]) for k in range(-2, 3)], np.uint8)[v.astype(int) + 2]
    scales = rng.integers(127, 130, (-(-rows // block), ref.ceil(cols))).astype(np.uint8)
    return Mat(env, rows, cols, block, e5m2, wide, more).put(codes, scales), ref.values(codes, scales, block, e5m2)


PRODUCTS = [(1, 1, 1), (1, 16, 16), (1, 300, 4096), (2, 129, 130), (3, 17, 127), (5, 64, 1000), (15, 257, 128), (16, 100, 640), (17, 33, 512),
            (31, 130, 300), (33, 200, 77), (64, 64, 64), (65, 500, 2049), (100, 127, 1), (127, 129, 257), (128, 128, 128), (129, 1, 333),
            (200, 300, 400), (256, 256, 256), (257, 513, 129), (300, 777, 1001), (513, 100, 3000), (1, 5000, 129), (5000, 3, 130), (640, 640, 640)]


@pytest.mark.parametrize("m,n,k", PRODUCTS, ids=["x".join(map(str, p)) for p in PRODUCTS])
@pytest.mark.parametrize("blocks", [(1, 1), (1, 128), (128, 128), (128, 1)], ids=["rows-rows", "rows-tiles", "tiles-tiles", "tiles-rows"])
def test_product_of_whole_numbers_is_exact(env, m, n, k, blocks):
    e5 = ((m + n) % 2 == 1, k % 3 == 0)
    a, va = whole_numbers(env, m, k, m + k, blocks[0], e5[0])
    b, vb = whole_numbers(env, n, k, n + k + 1, blocks[1], e5[1])
    want = va @ vb.T
    got = product(env, a, b, True)
    assert np.array_equal(got, want.astype(np.float32)), f"{(got != want).sum()} of {got.size} differ"
    got = product(env, a, b, False)
    assert np.array_equal(got, widen(bf16_bits(want.astype(np.float32))))


# tiles of 256 in bands of 64 rows, of 128 rows, whole, whole ones and bands of either; of 128; of 64 with the summed axis in parts;
# of 128 (into fp32) in parts
LARGE = [(1100, 2304, 1000), (2200, 2500, 1500), (5000, 5000, 130), (4100, 4200, 260), (4100, 5400, 260), (1500, 4096, 300), (300, 300, 8000), (2304, 768, 8192),
         (40, 3000, 8192), (20, 11008, 1000)]


@pytest.mark.parametrize("m,n,k", LARGE, ids=["x".join(map(str, p)) for p in LARGE])
@pytest.mark.parametrize("blocks", [(1, 128), (128, 1)], ids=["rows-tiles", "tiles-rows"])
def test_large_product_of_whole_numbers_is_exact(env, m, n, k, blocks):
    """Every tile shape, whole and cut by the edges, the workspace full of NaN before the call."""
    torch, dev = env
    a, va = whole_numbers(env, m, k, m + k, blocks[0], False)
    b, vb = whole_numbers(env, n, k, n + k + 1, blocks[1], k % 3 == 0)
    want = (torch.from_numpy(va).to(dev) @ torch.from_numpy(vb).to(dev).T).float().cpu().numpy()   # exact in 64 bits
    for f32 in (True, False):
        ws = torch.full((max(256, z.f8_product_workspace_bytes(a.m, b.m, z.F32 if f32 else 0)),), 0xFF, dtype=torch.uint8, device=dev)
        got = product(env, a, b, f32, ws=ws, ld_more=5)
        assert np.array_equal(got, want if f32 else widen(bf16_bits(want))), f"f32={f32}: {(got != want).sum()} of {got.size}"


def test_the_workspace_is_checked(env):
    torch, dev = env
    a, _ = whole_numbers(env, 300, 8000, 1, 1, False)
    b, _ = whole_numbers(env, 300, 8000, 2, 128, False)
    need = z.f8_product_workspace_bytes(a.m, b.m)
    assert need > 0
    d = torch.zeros(300, 300, dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device=dev)
    for bad, word in ((None, "NULL"), (ws[:need - 1], "needs"), (ws[8:], "256-byte")):
        with pytest.raises(z.Zero1Error) as e:
            z.f8_product(a.m, b.m, d, ws=bad)
        assert e.value.name == "ZERO1_EWORKSPACE" and word in e.value.message
    assert (d == 0).all()


@pytest.mark.parametrize("m,n,k", [(3, 200, 300), (130, 140, 260), (300, 520, 1100)])
def test_product_strides(env, m, n, k):
    a, va = whole_numbers(env, m, k, 1, 1, False, wide=16, more=4)
    b, vb = whole_numbers(env, n, k, 2, 128, False, wide=128 + 48, more=8)
    want = (va @ vb.T).astype(np.float32)
    for more in (1, 7, 8):
        assert np.array_equal(product(env, a, b, True, ld_more=more, skew=4), want)
        assert np.array_equal(product(env, a, b, False, ld_more=more, skew=2), widen(bf16_bits(want)))


@pytest.mark.parametrize("m,n,k", [(1, 1000, 4096), (16, 512, 2000), (40, 300, 1000), (129, 257, 5000), (512, 640, 1500)])
@pytest.mark.parametrize("e5a,e5b,blocks", [(False, False, (1, 128)), (True, False, (1, 1)), (True, True, (128, 128)), (False, True, (1, 1))])
def test_product_against_64_bits(env, m, n, k, e5a, e5b, blocks):
    """Operands as quantize makes them.  A product of two codes is exact in binary32; a sum of k of them takes at most
    k + k / 128 additions, each off by at most 2^-23 of the sum of magnitudes (2^-24 where it rounds to nearest; the
    matrix cores' own alignment may truncate): k 2^-22 of it covers both.  bf16: half of 2^-7 more."""
    xa, _ = source(env, m, k, m, True)
    xb, _ = source(env, n, k, n + 1, True)
    a = Mat(env, m, k, blocks[0], e5a).put(*ref.quantize(xa, blocks[0], e5a))
    b = Mat(env, n, k, blocks[1], e5b).put(*ref.quantize(xb, blocks[1], e5b))
    va, vb = (ref.values(*ref.quantize(x, bl, e), bl, e) for x, bl, e in ((xa, blocks[0], e5a), (xb, blocks[1], e5b)))
    want, mag = va @ vb.T, np.abs(va) @ np.abs(vb).T
    got = product(env, a, b, True).astype(np.float64)
    assert (np.abs(got - want) <= k * 2.0 ** -22 * mag).all()
    # and in the 2-norm by what rounding at random gives: the square root of the additions
    assert np.linalg.norm(got - want) <= 4 * k ** 0.5 * 2.0 ** -23 * np.linalg.norm(mag)
    got16 = product(env, a, b, False).astype(np.float64)
    assert (np.abs(got16 - want) <= k * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)).all()
    again = product(env, a, b, True)
    assert np.array_equal(again.view(np.uint32), got.astype(np.float32).view(np.uint32)), "a rerun gives the same bits"


def test_product_of_nan_and_extreme_scales(env):
    """NaN reaches its row of d, or its column, alone; scales over their whole range."""
    m, n, k = 40, 50, 256
    a, va = whole_numbers(env, m, k, 5, 1, False)
    b, vb = whole_numbers(env, n, k, 6, 1, False)
    ca, sa = (t.copy() for t in a.get())
    ca[7, 130] = 0x7F                                      # a NaN code
    sa[9, 1] = 255                                         # a NaN scale
    sa[11, :2] = 1
    sa[13, :2] = 240
    a.codes.put(ca.reshape(-1))
    a.scales.put(sa.reshape(-1))
    va = ref.values(ca[:, :k], sa[:, :2], 1, False)
    got = product(env, a, b, True)
    bad = np.zeros(m, bool)
    bad[[7, 9]] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    with np.errstate(all="ignore"):
        want = (va @ vb.T)[~bad].astype(np.float32)
        assert np.array_equal(got[~bad], want)
        got = product(env, a, b, False)
        assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], widen(bf16_bits(want)))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_product_at_the_ends_of_the_range(env, m):
    """Elements down to 2^-127 (fp32: bf16 holds them; 2^-136 counts as zero there), results below binary32's normal ones,
    and elements beyond 2^128 (fp32: infinite)."""
    n, k = 40, 128
    one, least, most = 0x38, 0x01, 0x7E
    for sa, sb, code, f32_zero, f32_inf in ((0, 127, one, 0, 0), (1, 110, one, 0, 0), (100, 20, one, 0, 0), (1, 127, least, 1, 0),
                                            (0, 254, most, 0, 1), (1, 1, most, 0, 0)):
        a = Mat(env, m, k).put(np.full((m, k), code, np.uint8), np.full((m, 1), sa, np.uint8))
        b = Mat(env, n, k).put(np.full((n, k), most if code == most else one, np.uint8), np.full((n, 1), sb, np.uint8))
        want = np.float32(k * ref.E4M3[code] * 2.0 ** (sa - 127) * ref.E4M3[most if code == most else one] * 2.0 ** (sb - 127))
        got = product(env, a, b, True)
        assert (got == (0.0 if f32_zero else np.inf if f32_inf else want)).all(), (sa, sb, got[0, 0], want)
        got = product(env, a, b, False)
        assert (got == widen(bf16_bits(np.array([want])))[0]).all(), (sa, sb, got[0, 0], want)


def test_rows_past_the_end_do_not_matter(env):
    """What lies behind the operands (guards of NaN codes) does not reach d."""
    for m, n, k in ((1, 3, 128), (130, 131, 384), (17, 250, 200)):
        va, vb = None, None
        rng = np.random.default_rng(1)
        a, b = Mat(env, m, k, fill=0x7F), Mat(env, n, k, fill=0x7F)
        ones = np.full((max(m, n), k), 0x38, np.uint8)     # 1.0
        a.put(ones[:m], np.full((m, ref.ceil(k)), 127, np.uint8))
        b.put(ones[:n], np.full((n, ref.ceil(k)), 127, np.uint8))
        assert (product(env, a, b, True) == k).all() and va is vb and rng is not None


def test_two_streams_and_a_captured_product(env):
    """Two products at once on two streams with workspaces of their own; and one captured, replayed between eager work
    on operands that change."""
    torch, dev = env
    shapes = [(5, 2000, 4096), (300, 300, 8000), (1, 512, 8192)]
    ops = [(whole_numbers(env, m, k, m, 1, False), whole_numbers(env, n, k, n, 128, False)) for m, n, k in shapes]
    streams = [torch.cuda.Stream() for _ in ops]
    ds = [torch.zeros(a.rows, b.rows, device=dev) for (a, _), (b, _) in ops]
    wss = [ws_tensor(torch, z.f8_product_workspace_bytes(a.m, b.m, z.F32), dev) for (a, _), (b, _) in ops]
    torch.cuda.synchronize()
    for _ in range(5):
        for ((a, _), (b, _)), d, w, s in zip(ops, ds, wss, streams):
            z.f8_product(a.m, b.m, d, flags=z.F32, ws=w, stream=s)
    torch.cuda.synchronize()
    for ((a, va), (b, vb)), d in zip(ops, ds):
        assert np.array_equal(d.cpu().numpy(), (va @ vb.T).astype(np.float32))
    for ((a, va), (b, vb)), d, w in zip(ops, ds, wss):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            z.f8_product(a.m, b.m, d, flags=z.F32, ws=w)
        for rep in range(3):
            c, s = (t.copy() for t in a.get())
            rng = np.random.default_rng(rep)
            s[:, :ref.ceil(a.cols)] = rng.integers(127, 130, (a.srows, ref.ceil(a.cols)))
            a.scales.put(s.reshape(-1))
            d.fill_(7.0)
            w.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            want = ref.values(c[:, :a.cols], s[:, :ref.ceil(a.cols)], 1, False) @ vb.T
            assert np.array_equal(d.cpu().numpy(), want.astype(np.float32))
        del graph


# ------------------------------------------------------------------ together
def test_layer_forward_backward_and_step(env):
    """A linear layer trained for two steps: its weight quantized both ways from the fp32 master, forward product, input
    gradient and weight gradient as products of the quantized tensors (the latter into the replica's flat
    gradient), the AdamW step with 8-bit moments on that; every intermediate against 64 bits or the oracle."""
    torch, dev = env
    tokens, n, k = 200, 140, 300
    rng = np.random.default_rng(8)
    w = (0.05 * rng.standard_normal((n, k))).astype(np.float32)
    S = n * k
    master = torch.from_numpy(w.reshape(-1).copy()).to(dev)
    param = torch.zeros(S, dtype=torch.bfloat16, device=dev)
    m, v = (torch.zeros(z.state8_bytes(S), dtype=torch.uint8, device=dev) for _ in range(2))
    pieces = [(S, 0, param, master, m, v)]
    table = ws_tensor(torch, z.mta_table_bytes(pieces), dev)
    plan = z.mta_plan(pieces, table, flags=z.MV_8BIT)
    ws = ws_tensor(torch, z.mta_workspace_bytes(plan, 1), dev)
    rsd = torch.zeros(1, dtype=torch.float64, device=dev)
    om, mm, vv = w.reshape(-1).copy(), np.zeros(S, np.float32), np.zeros(S, np.float32)
    st = [np.zeros(S, np.uint8), np.zeros(ref8.blocks(S), np.uint32)] * 2
    st = [a.copy() for a in st]
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=1.0)
    grad = torch.zeros(S, dtype=torch.bfloat16, device=dev)
    for t in (1, 2):
        x = widen(bf16_bits(rng.standard_normal((tokens, k)).astype(np.float32)))
        dy = widen(bf16_bits((1e-2 * rng.standard_normal((tokens, n))).astype(np.float32)))
        xs, dys = device_source(env, x, False), device_source(env, dy, False)
        qw, qwt = Mat(env, n, k, 128), Mat(env, k, n, 128)
        qx, qxt = Mat(env, tokens, k), Mat(env, k, tokens)
        qd, qdt = Mat(env, tokens, n, 1, True), Mat(env, n, tokens, 1, True)
        z.f8_quantize(master, n, k, q=qw.m, qt=qwt.m, flags=z.F32)
        z.f8_quantize(xs.view, tokens, k, q=qx.m, qt=qxt.m)
        z.f8_quantize(dys.view, tokens, n, q=qd.m, qt=qdt.m)
        wm = om.reshape(n, k)
        qw.check(wm, "w")
        qwt.check(np.ascontiguousarray(wm.T), "w^T")
        val = lambda q: ref.values(q.get()[0][:, :q.cols], q.get()[1][:, :ref.ceil(q.cols)], q.block, q.e5m2)   # noqa: E731
        assert np.array_equal(val(qw), val(qwt).T), "the weight and its transpose hold the same values"
        for a, b in ((qx, qw), (qd, qwt)):
            want, mag = val(a) @ val(b).T, np.abs(val(a)) @ np.abs(val(b)).T
            got = product(env, a, b, True)
            assert (np.abs(got - want) <= a.cols * 2.0 ** -22 * mag).all()
        z.f8_product(qdt.m, qxt.m, grad, ws=ws_tensor(torch, z.f8_product_workspace_bytes(qdt.m, qxt.m), dev))
        want, mag = val(qdt) @ val(qxt).T, np.abs(val(qdt)) @ np.abs(val(qxt)).T
        g = grad.view(torch.int16).cpu().numpy().view(np.uint16)
        assert (np.abs(widen(g).reshape(n, k) - want) <= tokens * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)).all()
        # close to the gradient of the layer before any rounding to 8 bits: each factor is off by 2^-4 and 2^-3 at most
        full = dy.T.astype(np.float64) @ x
        assert np.linalg.norm(want - full) <= (2.0 ** -3 + 2.0 ** -4) * np.linalg.norm(np.abs(dy).T.astype(np.float64) @ np.abs(x))
        z.mta_step([grad], 0, plan, dict(hp, step=t), rsd, 1, 0, ws=ws)
        mm, vv = ref8.decode(st[0], st[1], ref8.M), ref8.decode(st[2], st[3], ref8.V)
        op, rs = np.zeros(S, np.uint16), np.zeros(1)
        oracle.step([g], om, mm, vv, op, dict(hp, step=t), rs, 0)
        st = list(ref8.round_step(mm, np.sqrt(vv), st[1], st[3], 0))
        assert_f32_equal(master.cpu().numpy(), om, f"master t={t}")
        gc, gw = ref8.split(m.cpu().numpy(), S)
        assert np.array_equal(gc, st[0]) and np.array_equal(gw, st[1])
