"""e4m3 codes with a scale for each block of 128: equal to the rule's, bit for bit."""
import pytest
import torch

import train_reference as T

pytestmark = pytest.mark.gpu
B = T.B


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    return moe


def source(*shape, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp(3 * torch.randn((*shape[:-1], 1), generator=g, device="cuda"))
    v = (torch.randn(shape, generator=g, device="cuda") * size).to(torch.bfloat16)
    flat = v.view(-1, shape[-1])
    flat[0, :min(16, shape[-1])] = torch.tensor([0.0, -0.0, 448.0, 449.0, 450.0, 2.0 ** -9, 1.75 * 2.0 ** 20, 3e38, 1e-38, -1e-40,
                                                 0.875, 0.4375, -448.0, 17.0, 18.0, 19.0])[:min(16, shape[-1])].to(v)
    if flat.shape[0] > 2:
        flat[2] = 0
    return v


def same(q, s, want, name):
    assert torch.equal(s, want[1]), f"{name}: scales"
    assert torch.equal(q.view(torch.float8_e4m3fn).float(), want[0].view(torch.float8_e4m3fn).float()), f"{name}: codes"


@pytest.mark.parametrize("rows", [1, 2, 17, 1000, 5001])
@pytest.mark.parametrize("cols", [16, 112, 128, 144, 2064, 7168])
def test_rows(moe, rows, cols):
    v = source(rows, cols)
    same(*moe.moe_quantize_e4m3_block(v), T.quantize(v, 1, B), "rows")


@pytest.mark.parametrize("mats,rows,cols", [(1, 1, 16), (1, 128, 128), (3, 130, 272), (2, 768, 2048), (5, 1000, 144), (1, 4096, 7168)])
def test_tiles(moe, mats, rows, cols):
    v = source(mats, rows, cols)
    q, s = moe.moe_quantize_e4m3_block(v, block_rows=B)
    for m in range(mats):
        same(q[m], s[m], T.quantize(v[m], B, B), f"matrix {m}")


def test_matrices_of_rows(moe):
    v = source(3, 40, 272)
    q, s = moe.moe_quantize_e4m3_block(v)
    assert s.shape == (3, 40, 3)
    for m in range(3):
        same(q[m], s[m], T.quantize(v[m], 1, B), f"matrix {m}")


@pytest.mark.parametrize("counts", [[1], [128], [0, 0, 1, 0], [127, 129, 0, 256], [5000, 1, 300], [3] * 300, [0] * 1023 + [2]],
                         ids=lambda c: str(c[:4]))
@pytest.mark.parametrize("cols", [16, 144, 2064])
@pytest.mark.parametrize("extra", [0, 50])
def test_segments(moe, counts, cols, extra):
    rows = sum(counts) + extra
    v = source(rows, cols)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    m = moe.segment_rows(rows, len(counts))
    q = torch.full((rows, cols), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, T.blocks(cols)), 9.0, device="cuda")
    q_seg = torch.full((m, cols), 99, dtype=torch.uint8, device="cuda")
    s_seg = torch.full((m // B, cols), 9.0, device="cuda")
    ws = moe.workspace("combine")
    moe.moe_quantize_e4m3_segments(v, off, q=q, scale=s, q_seg=q_seg, scale_seg=s_seg, ws=ws)
    assert moe.read_device_error(ws) == 0
    n = sum(counts)
    same(q[:n], s[:n], T.quantize(v[:n], 1, B), "rows")
    assert (q[n:] == 99).all() and (s[n:] == 9).all()
    end = 0
    for e, a, b, pa, pb in T.spans(counts):
        if b > a:
            same(q_seg[pa:pa + b - a], s_seg[pa // B:pb // B], T.quantize(v[a:b], B, 1), f"segment {e}")
            assert (q_seg[pa + b - a:pb] == 0).all()
        end = pb
    assert (q_seg[end:] == 99).all() and (s_seg[end // B:] == 9).all()
    only = moe.moe_quantize_e4m3_segments(v, off, both=False, ws=ws)
    assert only[0] is None and only[1] is None
    assert torch.equal(only[2][:end], q_seg[:end]) and torch.equal(only[3][:end // B], s_seg[:end // B])


def test_one_segment_needs_no_offsets(moe):
    v = source(300, 272)
    q, s, q_seg, s_seg = moe.moe_quantize_e4m3_segments(v, None)
    same(q, s, T.quantize(v, 1, B), "rows")
    same(q_seg[:300], s_seg, T.quantize(v, B, 1), "segment")
    assert (q_seg[300:] == 0).all()


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, 4, 8, 11], [1, 4, 8, 9], [0, -2, 8, 9]], ids=str)
def test_bad_offsets_write_nothing(moe, bad):
    v = source(9, 128)
    ws = moe.workspace("combine")
    q_seg = torch.full((moe.segment_rows(9, 3), 128), 99, dtype=torch.uint8, device="cuda")
    s_seg = torch.full((q_seg.shape[0] // B, 128), 9.0, device="cuda")
    moe.moe_quantize_e4m3_segments(v, torch.tensor(bad, dtype=torch.int32, device="cuda"), both=False, q_seg=q_seg,
                                   scale_seg=s_seg, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert (q_seg == 99).all() and (s_seg == 9).all()


def test_infinities_saturate_and_nan_stays(moe):
    """As in the row quantiser; the other blocks do not notice."""
    v = source(256, 256)
    clean = T.quantize(v, 1, B)
    v[4, 3], v[4, 5] = float("inf"), float("-inf")
    v[6, 130] = float("nan")
    q, _ = moe.moe_quantize_e4m3_block(v)
    got = q.view(torch.float8_e4m3fn).float()
    assert got[4, 3] == 448 and got[4, 5] == -448 and got[6, 130].isnan()
    keep = torch.ones((256, 256), dtype=torch.bool, device="cuda")
    keep[4, :B], keep[6, B:] = False, False
    assert torch.equal(got[keep], clean[0].view(torch.float8_e4m3fn).float()[keep])
    qs = moe.moe_quantize_e4m3_segments(v, None, both=False)[2].view(torch.float8_e4m3fn).float()
    assert qs[4, 3] == 448 and qs[4, 5] == -448 and qs[6, 130].isnan()
    qt = moe.moe_quantize_e4m3_block(v, block_rows=B)[0].view(torch.float8_e4m3fn).float()
    assert qt[4, 3] == 448 and qt[4, 5] == -448 and qt[6, 130].isnan()


def test_agrees_with_the_row_quantiser_on_one_block(moe):
    v = source(64, 128)
    q, s = moe.moe_quantize_e4m3_block(v)
    rq, rs = moe.moe_quantize_e4m3(v)
    assert torch.equal(q, rq) and torch.equal(s[:, 0], rs)
