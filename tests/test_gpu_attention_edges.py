"""The attention operators at the edges of their ranges: rounding into E4M3 pages,
weights far apart, values that are not finite, page ids, windows, token offsets and
streams.  Bounds as in tests/_attention_reference.py unless a test says otherwise."""
import math

import pytest
import torch

import _attention_reference as ref
from test_gpu_attention import BAD_INDEX, DEV, Paged, _within, nb  # noqa: F401

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ append --
def _appended(nb, x, scale):
    """Bytes of an E4M3 cache after x [T, H, D] went in as keys and as values, one
    request from position 0 on."""
    T, H, D = x.shape
    page = 16
    pages = -(-T // page)
    kc, vc = (torch.zeros(pages, page, H, D, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    sc = scale.to(DEV)
    cache = nb.PagedKVCache(kc, vc, k_scale=sc, v_scale=sc)
    batch = nb.AttnBatch(_i32(0, T), _i32(T), torch.arange(pages, dtype=torch.int32, device=DEV)[None],
                         max_new=T)
    ws = nb.attn_workspace()
    nb.kv_append(cache, batch, x.to(DEV), x.to(DEV), ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    return [c.view(torch.uint8).flatten(0, 1)[:T].cpu() for c in (kc, vc)]


@pytest.mark.parametrize("D", [64, 128])
def test_kv_append_divides_by_the_scale(nb, D):
    """The stored byte is that of the fp32 quotient, ties included: scales for which
    quotients fall on or beside the middle between two E4M3 numbers, where a product
    with the rounded reciprocal goes to the other side, and the ends of the range, where
    the reciprocal is infinite or subnormal."""
    ties = torch.arange(17, 32, 2).float()
    tops = torch.arange(128, 256).float()
    scale = torch.cat([(tops[:, None] / ties).flatten()[::23], torch.tensor(
        [7.0, 1e-39, 2.0 ** -149, 2.0 ** -128, 3e38, 1.0])])
    H = scale.numel()
    x = torch.cat([tops, -tops, tops * 2.0 ** -9, torch.zeros(64), 7 * ties,
                   torch.tensor([2.0 ** -126, -2.0 ** -126, 2.0 ** -133, 3e38, -3e38])])
    x = torch.nn.functional.pad(x, (0, -x.numel() % D)).view(-1, 1, D).expand(-1, H, D)
    x = x.bfloat16().contiguous()
    quotient = (x.float() / scale[:, None]).clamp(-448, 448)
    want = quotient.to(torch.float8_e4m3fn).view(torch.uint8)
    other = (x.float() * (1 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert (other.view(torch.uint8)[:, :-6] != want[:, :-6]).sum() > 9    # the cases are there
    for got in _appended(nb, x, scale):
        assert torch.equal(got, want)
