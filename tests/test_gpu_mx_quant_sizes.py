"""MX quantisation and its inverse of inputs that take more than the 2^32 threads
of one launch: turned weights of very many of the smallest experts (a workgroup
each), and more than 2^36 values in rows (4096 a workgroup)."""
import pytest
import torch

from quantized_moe_grouped_amd import binding as B

pytestmark = pytest.mark.gpu


def _bytes(t):
    return t.view(torch.uint8)


def _needs(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def _repeated(small, copies):
    """`small` copies times over, without its like in temporary memory."""
    x = torch.empty((copies, *small.shape), dtype=small.dtype, device="cuda")
    x[0] = small
    done = 1
    while done < copies:
        more = min(done, copies - done)
        x[done:done + more] = x[:more]
        done += more
    return x


def test_turned_weights_of_very_many_experts():
    _needs(40)
    e = 2 ** 24 + 5
    small = torch.randn((64, 8), device="cuda").bfloat16()
    x = _repeated(small, e)
    codes, scales = B.mx_quantize(x, transpose=True)
    c, s = B.mx_quantize(small[None], transpose=True)
    for part in (slice(0, 3), slice(2 ** 23 - 2, 2 ** 23 + 2), slice(2 ** 24 - 2, e)):
        assert (_bytes(codes[part]) == _bytes(c)).all() and (_bytes(scales[part]) == _bytes(s)).all(), part


def test_rows_of_very_many_values():
    _needs(200)
    k = 8192
    small = torch.randn((1024, k), device="cuda").bfloat16()
    copies = 2 ** 36 // small.numel() + 1
    x = _repeated(small, copies).view(-1, k)
    codes, scales = B.mx_quantize(x, format="fp4")
    c, s = B.mx_quantize(small, format="fp4")
    rows = x.shape[0]
    parts = [slice(a, a + 1024) for a in (0, (rows // 2048) * 1024, rows - 1024)]
    for part in parts:
        assert torch.equal(_bytes(codes)[part], _bytes(c)) and torch.equal(_bytes(scales)[part], _bytes(s)), part
    del x
    torch.cuda.empty_cache()
    back, want = B.mx_dequantize(codes, scales), B.mx_dequantize(c, s)
    for part in parts:
        assert torch.equal(back[part], want), part
