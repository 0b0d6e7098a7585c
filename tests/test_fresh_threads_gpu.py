"""The first CUDA call that a thread makes may be any of the library's: a thread without a current context, whose outputs
come from memory that torch has cached, gets what the main thread gets."""
import threading

import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_paged_attention_gpu import fill, queries
from test_paged_cache_gpu import make, qkv

pytestmark = pytest.mark.gpu


def in_a_thread(call):
    got = []

    def work():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def rand(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("max_new", [1, 100])
def test_serving(max_new):
    new, held = [1, 2, 1], [300, 200, 40]
    cache, batch, starts, N = make(new, held, 2, 64, 16, "heads")
    fill(cache, batch, held)
    q, k, v = qkv(N, 4, 2, 64)
    r = tll.Rotary(64)
    turned = tll.cache_append(q, k, v, cache, batch, rotary=r)
    out = tll.paged_attention(turned, cache, batch, max_new=max_new)
    buf = torch.empty_like(out), torch.empty_like(out)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.paged_attention(turned, cache, batch, max_new=max_new, out=buf[0])), out)
    assert torch.equal(in_a_thread(lambda: tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=buf[1])), turned)
    positions = torch.arange(N, device="cuda")
    want = tll.rotary_forward(q, positions, r)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.rotary_forward(q, positions, r, out=buf[0])), want)


@pytest.mark.parametrize("M,dtype,precision", [(64, torch.bfloat16, "bf16"), (8, torch.bfloat16, "bf16"),
                                               (64, torch.float32, "tf32"), (64, torch.float32, "fp32")])
def test_products(M, dtype, precision):
    x, w = rand(M, 256, dtype=dtype), rand(192, 256, dtype=dtype, seed=1)
    want = tll.forward(x, w, precision=precision)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.forward(x, w, precision=precision, out=out)), want)
    dx = tll.backward_data(want, w, precision=precision)
    got = torch.empty_like(dx)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.backward_data(want, w, precision=precision, out=got)), dx)


def test_attention():
    x = rand(2 * 70, 3 * 128)
    want, lse = tll.attention_forward(x, 2, 70, 2, with_lse=True)
    out, d = torch.empty_like(want), torch.empty_like(x)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.attention_forward(x, 2, 70, 2, out=out)), want)
    grad = tll.attention_backward(x, want, lse, want, 2, 70, 2)
    torch.cuda.synchronize()
    assert torch.equal(in_a_thread(lambda: tll.attention_backward(x, want, lse, want, 2, 70, 2, dqkv=d)), grad)
