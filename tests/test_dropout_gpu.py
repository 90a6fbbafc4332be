"""rc_dropout and rc_all_reduce_dropout against the definition in the header,
bit for bit: the Philox4x32-10 blocks in 64-bit integers, binary32 arithmetic
with one rounding per operation, the all-reduce's ring order."""
import numpy as np
import pytest
import torch

import rc_inputs
from util import assert_bits, check_canary, empty_dev, to_dev, to_host

pytestmark = pytest.mark.gpu
ESZ = {"f32": 4, "bf16": 2}


@pytest.fixture(scope="module")
def rc():
    import collective_rc_all_b200 as m
    assert torch.cuda.is_available()
    return m


def philox(block, seed):
    """Philox4x32-10 of counters (block, 0): four arrays of 32-bit words."""
    m32, lo = np.uint64(32), np.uint64(0xFFFFFFFF)
    c = [block & lo, block >> m32, np.zeros_like(block), np.zeros_like(block)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        u, v = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(v >> m32) ^ c[1] ^ np.uint64(k[0]), v & lo, (u >> m32) ^ c[3] ^ np.uint64(k[1]), u & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(first, n, seed, prob):
    e = np.uint64(first) + np.arange(n, dtype=np.uint64)   # wraps modulo 2^64
    w = np.stack(philox(e >> np.uint64(3), seed), 1)
    lane = (e & np.uint64(7)).astype(np.int64)
    half = w[np.arange(n), lane // 2] >> (16 * (lane % 2)).astype(np.uint64) & np.uint64(0xFFFF)
    return half.astype(np.int64) >= int(np.rint(prob * 65536))


def factor(prob, scale):
    t = int(np.rint(prob * 65536))
    return np.float32(np.float64(np.float32(scale)) * (65536.0 / (65536.0 - t))) if t < 65536 else np.float32(0)


def widen(x, dt):
    return x if dt == "f32" else (x.astype(np.uint32) << 16).view(np.float32)


def narrow(x, dt):
    return x if dt == "f32" else torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def expect(xs, res, n, dt, prob, seed, offset, stride, scale):
    out = []
    for r, x in enumerate(xs):
        k = keep((offset + r * stride) % 2**64, n, seed, prob)
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.where(k, widen(x, dt) * factor(prob, scale), np.float32(0))
            if res is not None:
                y = widen(res[r], dt) + y
        out.append(narrow(y.astype(np.float32), dt))
    return out


def test_known_generator_blocks():
    """The generator's published test vectors (Random123, philox4x32 10 rounds)
    that this counter layout can reach: counter 0, key 0."""
    w = [int(x[0]) for x in philox(np.zeros(1, np.uint64), 0)]
    assert w == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 4099, 100003])
@pytest.mark.parametrize("p,stride", [(1, 0), (3, None), (16, 8)])
@pytest.mark.parametrize("res", [False, True])
def test_dropout_matches_definition(rc, dt, n, p, stride, res):
    stride = n if stride is None else stride
    prob, seed, offset = 0.3, 0x123456789ABCDEF1, 5 * n + 3
    xs = rc_inputs.normal(p, n, seed=n + p, dt=dt)
    rs = rc_inputs.normal(p, n, seed=n + p + 1, dt=dt) if res else None
    d, _ = to_dev(xs, dt)
    e = to_dev(rs, dt)[0] if res else None
    y, back = empty_dev(n, dt, p)
    rc.rc_dropout(d, y, prob, seed, offset=offset, rank_stride=stride, residual=e, scale=0.5)
    torch.cuda.synchronize()
    want = expect(xs, rs, n, dt, prob, seed, offset, stride, 0.5)
    for r in range(p):
        assert_bits(to_host(y[r], dt), want[r], f"rank {r}")
    check_canary(back, n * ESZ[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 4, 6, 2**64 - 100, 2**40 + 2])
def test_every_phase_of_the_index_and_misaligned_buffers(rc, dt, offset):
    n, p, seed = 1000, 2, 2**64 - 3
    xs = rc_inputs.normal(p, n, seed=3, dt=dt)
    want = expect(xs, xs, n, dt, 0.5, seed, offset, 17, 1.0)
    for shift in (0, 16, ESZ[dt]):
        d, _ = to_dev(xs, dt, offset_bytes=shift)
        e, _ = to_dev(xs, dt, offset_bytes=shift)
        y, back = empty_dev(n, dt, p, offset_bytes=shift)
        rc.rc_dropout(d, y, 0.5, seed, offset=offset, rank_stride=17, residual=e)
        torch.cuda.synchronize()
        for r in range(p):
            assert_bits(to_host(y[r], dt), want[r], f"shift {shift} rank {r}")
        check_canary(back, shift + n * ESZ[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("prob", [0.0, 1e-6, 0.999, 0.99999999, 1.0])
def test_probability_edges_and_non_finite_values(rc, dt, prob):
    n = 777
    x = rc_inputs.normal(1, n, seed=1, dt="f32")[0]
    x[::5], x[1::5], x[2::5] = np.inf, -np.inf, np.nan
    x = narrow(x, dt)
    d, _ = to_dev([x], dt)
    y, _ = empty_dev(n, dt, 1)
    rc.rc_dropout(d, y, prob, 11)
    torch.cuda.synchronize()
    got, want = widen(to_host(y[0], dt), dt), widen(expect([x], None, n, dt, prob, 11, 0, 0, 1.0)[0], dt)
    assert np.array_equal(got, want, equal_nan=True)
    k = keep(0, n, 11, prob)
    assert np.all(got[~k] == 0)                       # a dropped NaN is zero
    if prob in (0.0, 1e-6):
        assert k.all()
    if prob in (0.99999999, 1.0):
        assert not k.any()


def test_in_place_and_backward_is_the_same_mask(rc):
    n, p, prob, seed = 5003, 4, 0.4, 99
    xs = rc_inputs.normal(p, n, seed=8, dt="f32")
    d, _ = to_dev(xs, "f32")
    rc.rc_dropout(d, d, prob, seed, offset=24, rank_stride=n)
    g, _ = to_dev([np.ones(n, np.float32)] * p, "f32")
    rc.rc_dropout(g, g, prob, seed, offset=24, rank_stride=n)
    torch.cuda.synchronize()
    for r in range(p):
        assert_bits(to_host(d[r], "f32"), expect(xs, None, n, "f32", prob, seed, 24 + r * n, 0, 1.0)[r], "y")
        k = keep(24 + r * n, n, seed, prob)
        assert_bits(to_host(g[r], "f32"), np.where(k, factor(prob, 1.0), np.float32(0)), "dx")


def test_keep_rate_and_ranks_differ(rc):
    """Share of kept elements within 6 standard deviations; masks of two ranks
    with their own index ranges agree as often as independent ones."""
    n, prob = 1 << 20, 0.25
    x = [torch.ones(n, device="cuda") for _ in range(2)]
    rc.rc_dropout(x, x, prob, 5, rank_stride=n)
    k = [(t != 0).double() for t in x]
    sd = (prob * (1 - prob) / n) ** 0.5
    for t in k:
        assert abs(float(t.mean()) - (1 - prob)) < 6 * sd
    agree, q = float((k[0] == k[1]).double().mean()), (1 - prob) ** 2 + prob ** 2
    assert abs(agree - q) < 6 * (q * (1 - q) / n) ** 0.5


def ring_fold(xs, n, p):
    C = -(-n // p)
    out = np.empty(n, np.float32)
    for c in range(p):
        s = slice(c * C, min(n, (c + 1) * C))
        acc = xs[(c + 1) % p][s].copy()
        for k in range(1, p):
            acc = acc + xs[(c + 1 + k) % p][s]
        out[s] = acc
    return out


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("p", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("n", [1, 13, 4096, 30011])
@pytest.mark.parametrize("res", [False, True])
def test_all_reduce_dropout(rc, dt, p, n, res):
    prob, seed, offset = 0.2, 77, 12345
    xs = rc_inputs.normal(p, n, seed=n * p, dt=dt)
    rs = rc_inputs.normal(p, n, seed=n * p + 1, dt=dt) if res else None
    total = ring_fold([widen(x, dt) for x in xs], n, p)
    k = keep(offset, n, seed, prob)
    v = np.where(k, total * factor(prob, 0.25), np.float32(0))
    for shift in (0, 16, ESZ[dt]):
        d, _ = to_dev(xs, dt, offset_bytes=shift)
        e = to_dev(rs, dt, offset_bytes=shift)[0] if res else None
        y, back = empty_dev(n, dt, p, offset_bytes=shift)
        rc.rc_all_reduce_dropout(d, y, prob, seed, offset=offset, residual=e, scale=0.25)
        torch.cuda.synchronize()
        for r in range(p):
            want = narrow((widen(rs[r], dt) + v if res else v).astype(np.float32), dt)
            assert_bits(to_host(y[r], dt), want, f"shift {shift} rank {r}")
        check_canary(back, shift + n * ESZ[dt])


def test_all_reduce_dropout_in_place_and_without_dropping(rc):
    """prob 0 and no residual is the all-reduce, in place too."""
    p, n = 8, 8192 + 24
    xs = rc_inputs.normal(p, n, seed=2, dt="bf16")
    a, _ = to_dev(xs, "bf16")
    b, _ = to_dev(xs, "bf16")
    rc.rc_all_reduce_dropout(a, a, 0.0, 1)
    rc.rc_all_reduce(b, b)
    torch.cuda.synchronize()
    for r in range(p):
        assert_bits(to_host(a[r], "bf16"), to_host(b[r], "bf16"), f"rank {r}")


def test_captured_and_replayed(rc):
    n, p = 10000, 2
    x = [torch.randn(n, device="cuda") for _ in range(p)]
    y, z = [torch.empty_like(t) for t in x], [torch.empty_like(t) for t in x]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rc.rc_all_reduce_dropout(x, y, 0.1, 3)
        rc.rc_dropout(y, z, 0.1, 4)
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t in x:
            t.normal_()
        g.replay()
        want = [torch.empty_like(t) for t in x]
        rc.rc_all_reduce_dropout(x, want, 0.1, 3)
        rc.rc_dropout(want, want, 0.1, 4)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(z, want))
