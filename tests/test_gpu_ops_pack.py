"""Packing to 8 bits with a scale for every 128 elements, and back, on the GPU: bit for bit
what the definition in 64 bits gives (x times a power of two is exact, and one rounding
follows)."""
import pytest
import torch

import ops_scaled_common as sc
import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = [(1, 1), (1, 300), (300, 1), (2, 127), (128, 128), (129, 257), (64, 1600), (1000, 33), (385, 641), (2049, 515)]


def make(rows, width, t, seed=0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(rows, width + pad, dtype=t, device=DEV)[:, :width]
    x.copy_(torch.randn(rows, width, generator=g, device=DEV) * torch.exp(2 * torch.randn(rows, 1, generator=g, device=DEV)))
    return x


def room(rows, width, square, pad=0):
    shape = (-(-rows // 128) if square else rows, -(-width // 128))
    codes = torch.full((rows, width + pad), 0x55, dtype=torch.uint8, device=DEV)
    exps = torch.full((shape[0], shape[1] + pad), 0x55, dtype=torch.uint8, device=DEV)
    return codes.view(torch.float8_e4m3fn)[:, :width], exps[:, :shape[1]]


def expected(x, square):
    x = x.double()
    top = 1.875 * 2.0 ** 127             # (no finite number becomes infinite)
    x = torch.where(torch.isfinite(x), x.clamp(-top, top), x)
    _, big = sc.blocks_of(x, square)
    E = sc.scale_byte(big)
    return sc.codes(x / torch.exp2(sc.spread(E.double(), *x.shape, square) - 127)), E


def same(codes, exps, x, square):
    want, E = expected(x, square)
    got = codes.view(torch.uint8).long()
    nan = (want & 127) == 127
    assert torch.equal(exps.long(), E)
    assert torch.equal((got & 127) == 127, nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("rows,width", SIZES)
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("square", [False, True])
def test_both_ways(rows, width, kind, square):
    x = make(rows, width, TYPES[kind], seed=rows + width, pad=3)
    c, e = room(rows, width, square, 2)
    ct, et = room(width, rows, square, 1)
    zs.zero_scaled_pack(x, c, e, ct, et)
    same(c, e, x, square)
    same(ct, et, x.t(), square)
    if square:
        assert torch.equal(c.view(torch.uint8).t(), ct.view(torch.uint8)) and torch.equal(e.t(), et)
    for codes, exps in ((c, e), (ct, et)):
        for t in TYPES.values():
            out = torch.empty(codes.shape, dtype=t, device=DEV)
            zs.zero_scaled_unpack(codes, exps, out)
            want = sc.values(codes, exps, square)
            assert torch.equal(out, want.to(torch.float32).to(t))
            if t != torch.float16:
                assert torch.equal(out.double(), want)
    # one of them alone has the same bits
    c2, e2 = room(rows, width, square)
    ct2, et2 = room(width, rows, square)
    zs.zero_scaled_pack(x, c2, e2)
    zs.zero_scaled_pack(x, codes_t=ct2, exps_t=et2)
    for a, b in ((c, c2), (ct, ct2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(e, e2) and torch.equal(et, et2)


def test_every_code_and_every_tie():
    """All magnitudes of the format, the middles between them, and numbers next to both,
    beside one that settles the scale."""
    table = sc.E4M3.to(DEV).float()
    mids = (table[1:] + table[:-1]) / 2
    near = torch.cat([z * (1 + s * 2.0 ** -20) for z in (table, mids) for s in (-1, 0, 1)])
    near = near[near <= 448]
    near = torch.cat([near, -near])
    near = torch.nn.functional.pad(near, (0, -near.numel() % 127)).view(-1, 127)
    x = torch.cat([torch.full((near.shape[0], 1), 448.0, device=DEV), near], 1)
    for by in (1.0, 2.0 ** -50, 2.0 ** 100):
        c, e = room(*x.shape, False)
        zs.zero_scaled_pack(x * by, c, e)
        same(c, e, x * by, False)


def test_the_range_of_scales():
    x = torch.randn(60, 128, device=DEV).clamp(-3, 3)
    x[:, 0] = 4.0
    x = torch.ldexp(x, torch.arange(-150, 150, 5, device=DEV)[:, None]).clamp(-3e38, 3e38)
    x[7] = 0
    x[8, 1:] = 0
    x[9] = 3.4028234663852886e38
    for square in (False, True):
        c, e = room(60, 128, square)
        zs.zero_scaled_pack(x, c, e)
        same(c, e, x, square)
        out = torch.empty(60, 128, dtype=torch.bfloat16, device=DEV)
        zs.zero_scaled_unpack(c, e, out)
        assert torch.equal(out.double(), sc.values(c, e, square))
    # the mantissa at which the next scale is taken
    edge = torch.zeros(4, 128, device=DEV)
    edge[0, 5], edge[1, 5], edge[2, 5], edge[3, 5] = 1.75, 1.75 * (1 + 2.0 ** -23), 2.0, 1.7499
    c, e = room(4, 128, False)
    zs.zero_scaled_pack(edge, c, e)
    assert e[:, 0].tolist() == [119, 120, 120, 119]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
def test_what_is_not_finite(kind):
    x = make(200, 300, TYPES[kind], seed=3)
    x[3, 7], x[150, 290], x[20, 20] = float("inf"), float("-inf"), float("nan")
    x[5, :128] = float("inf")
    for square in (False, True):
        c, e = room(200, 300, square)
        ct, et = room(300, 200, square)
        zs.zero_scaled_pack(x, c, e, ct, et)
        same(c, e, x, square)
        same(ct, et, x.t(), square)
        out = torch.empty(200, 300, device=DEV)
        zs.zero_scaled_unpack(c, e, out)
        assert torch.equal(torch.isnan(out), ~torch.isfinite(x))


def test_every_byte_of_a_scale():
    c = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1).view(torch.float8_e4m3fn)
    e = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 2)
    out = torch.empty(256, 256, device=DEV)
    zs.zero_scaled_unpack(c, e, out)
    want = sc.values(c, e, False).float()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], want[~nan])


def test_nothing_around_is_written_and_nothing_of_nothing():
    x = make(70, 150, torch.float32, seed=1, pad=9)
    big, be = torch.full((70, 200), 9, dtype=torch.uint8, device=DEV), torch.full((70, 4), 9, dtype=torch.uint8, device=DEV)
    zs.zero_scaled_pack(x, big.view(torch.float8_e4m3fn)[:, 1:151], be[:, 1:3])
    assert (big[:, 0] == 9).all() and (big[:, 151:] == 9).all() and (be[:, 0] == 9).all() and (be[:, 3] == 9).all()
    same(big.view(torch.float8_e4m3fn)[:, 1:151], be[:, 1:3], x, False)
    out = torch.full((70, 170), 5.0, device=DEV)
    zs.zero_scaled_unpack(big.view(torch.float8_e4m3fn)[:, 1:151], be[:, 1:3], out[:, 7:157])
    assert (out[:, :7] == 5).all() and (out[:, 157:] == 5).all()
    for shape in ((0, 5), (5, 0)):
        c, e = room(*shape, False)
        zs.zero_scaled_pack(torch.empty(shape, device=DEV), c, e)
        zs.zero_scaled_unpack(c, e, torch.empty(shape, device=DEV))


def test_graph_and_stream():
    x = make(1111, 777, torch.bfloat16, seed=2)
    c, e = room(1111, 777, False)
    ct, et = room(777, 1111, False)
    out = torch.empty(1111, 777, device=DEV)

    def both(stream=None):
        zs.zero_scaled_pack(x, c, e, ct, et, stream=stream)
        zs.zero_scaled_unpack(c, e, out, stream=stream)

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in range(3):
        x.mul_(-1.7)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(c, e, x, False)
        same(ct, et, x.t(), False)
        assert torch.equal(out.double(), sc.values(c, e, False))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x2 = out.clone()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    assert torch.equal(out, x2)


def test_refusals():
    x = torch.zeros(200, 300, device=DEV)
    c, e = room(200, 300, False)
    ct, et = room(300, 200, True)
    with pytest.raises(ValueError, match="squares"):
        zs.zero_scaled_pack(x, c, e, ct, et)
    with pytest.raises(ValueError, match="shape"):
        zs.zero_scaled_pack(x, c, e[:, :2])
    with pytest.raises(TypeError, match="float8"):
        zs.zero_scaled_pack(x, c.view(torch.uint8), e)
    with pytest.raises(zs.ZeroError, match="both or neither"):
        zs.zero_scaled_pack(x, c)
    with pytest.raises(zs.ZeroError, match="both NULL"):
        zs.zero_scaled_pack(x)
