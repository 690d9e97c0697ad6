"""e2f_checkpoint_store and e2f_checkpoint_load: codes, scale bytes and decoded values equal the plain 64-bit
implementation exactly."""
import pytest
import torch

import atomistic_cell_list_b200 as e2f
import feature_ref as R

pytestmark = pytest.mark.gpu


def _values(rows, C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, C, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    return x.to(R.DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 1), (3, 5), (7, 31), (5, 32), (64, 33), (40, 64), (9, 100), (200, 128), (3, 255),
                                    (12, 256), (2, 1000), (3, 4097), (1, 20000)])
def test_codes_and_values(rows, C, dtype):
    x = _values(rows, C, dtype, seed=C)
    val, code, byte = R.coded(x)
    codes, scales = e2f.e2f_checkpoint_store(x.cuda())
    assert torch.equal(codes.cpu(), code) and torch.equal(scales.cpu(), byte)
    assert torch.equal(e2f.e2f_checkpoint_load(codes, scales).cpu().double(), val)
    assert torch.equal(e2f.e2f_checkpoint_load(codes, scales, "bf16").cpu().double(), val)


def test_extreme_values():
    vals = [0.0, -0.0, 1e-45, 1.2e-38, 2.0 ** -126, 2.0 ** -120, 2.0 ** -119, 3.4e38, -3.4e38, 1.9999999, 127.5, 2.0 ** 127]
    x = torch.tensor([[v] + [v * 0.3, -v * 0.7] + [0.0] * 29 for v in vals], dtype=torch.float32)
    val, code, byte = R.coded(x)
    codes, scales = e2f.e2f_checkpoint_store(x.cuda())
    assert torch.equal(codes.cpu(), code) and torch.equal(scales.cpu(), byte)
    assert torch.equal(e2f.e2f_checkpoint_load(codes, scales).cpu().double(), val)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_block_with_a_non_finite_value_is_nan(bad):
    x = _values(4, 100, "f32")
    x[2, 70] = bad
    val, _, byte = R.coded(x)
    codes, scales = e2f.e2f_checkpoint_store(x.cuda())
    assert torch.equal(scales.cpu(), byte)
    got = e2f.e2f_checkpoint_load(codes, scales).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(val)) and torch.equal(got.nan_to_num(), val.nan_to_num())


def test_every_scale_byte_decodes():
    """A checkpoint written elsewhere: all 255 exponents and codes -128..127, as code 2^(s - 133) in fp32."""
    codes = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 8)
    got = e2f.e2f_checkpoint_load(codes.cuda(), scales.cuda()).cpu()
    want = torch.ldexp(codes.double(), scales[:, :1].int() - 133).float()
    assert torch.isnan(got[255]).all() and torch.equal(got[:255], want[:255])


def test_shapes_streams_capture_and_rows_behind():
    x = _values(24, 96, "bf16").view(2, 12, 96).cuda()
    codes, scales = e2f.e2f_checkpoint_store(x)
    assert codes.shape == (2, 12, 96) and scales.shape == (2, 12, 3)
    big = {"codes": torch.full((3, 12, 96), 77, dtype=torch.int8, device="cuda"),
           "scales": torch.full((3, 12, 3), 77, dtype=torch.uint8, device="cuda")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e2f.e2f_checkpoint_store(x, out={k: v[:2] for k, v in big.items()}, stream=s)
    got = e2f.e2f_checkpoint_load(big["codes"][:2], big["scales"][:2], "bf16", stream=s)
    s.synchronize()
    assert torch.equal(big["codes"][:2], codes) and torch.equal(big["scales"][:2], scales)
    assert (big["codes"][2:] == 77).all() and (big["scales"][2:] == 77).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        back = e2f.e2f_checkpoint_load(*e2f.e2f_checkpoint_store(x), "bf16")
    x.copy_(_values(24, 96, "bf16", seed=4).view(2, 12, 96))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, e2f.e2f_checkpoint_load(*e2f.e2f_checkpoint_store(x), "bf16"))
    assert not torch.equal(back, got)
    empty = torch.zeros(0, 5, device="cuda")
    assert e2f.e2f_checkpoint_load(*e2f.e2f_checkpoint_store(empty)).shape == (0, 5)
    with pytest.raises(ValueError):
        e2f.e2f_checkpoint_load(codes, scales[..., :2])
