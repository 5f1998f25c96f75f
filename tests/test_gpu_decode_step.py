"""The operators as a serving step and a training step use them: the new tokens' keys and values come out of the
matrix-vector product, go through the paged cache and back, the tokens are routed, and the experts' two products
with the routing weights make the MoE layer's output; the router's balance loss runs on the same routing."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import balance as B
from oracle import cache as C
from oracle import moe as M
from oracle import matvec as V
from oracle import quant as Q
from tests.gpu_common import assert_moe_close, bf16_dev, bf16_host_bits, bf16_host_f64, gpu_standard_weights

pytestmark = pytest.mark.gpu


def moe_by_products(x, logits, w13, s13, w2, s2, b13, b2, k):
    ids, w, offs, sp = mx.route(logits, k)
    h = mx.fp4_expert_matvec(x, w13, s13, offs, sp, b13, top_k=k, swiglu=True)
    o = mx.fp4_expert_matvec(h, w2, s2, offs, sp, b2, out_dtype=torch.float32)
    return ids, (o.view(*ids.shape, -1) * w[:, :, None]).sum(1).bfloat16()


def test_tiny_layer_equals_the_moe_layer_and_the_oracle():
    cfg = synth.MOE_CONFIGS["tiny"]
    x_bits, logits = synth.moe_activations(cfg)
    w13, s13, w2, s2, b13, b2 = gpu_standard_weights(cfg)
    x, lg = bf16_dev(x_bits), torch.from_numpy(logits).cuda()
    ids, y = moe_by_products(x, lg, w13, s13, w2, s2, b13, b2, cfg.k)
    y_ref, _, _ = M.moe_ref(x_bits, logits, cfg.k, w13.cpu().numpy(), s13.cpu().numpy(), w2.cpu().numpy(), s2.cpu().numpy(),
                            bf16_host_bits(b13), bf16_host_bits(b2))
    # the layer's own tolerance covers one rounding of the SwiGLU output to bf16, 2^-9 of it on average over I
    assert_moe_close(bf16_host_f64(y), y_ref, None, "products")
    assert_moe_close(bf16_host_f64(mx.MoE(w13, s13, w2, s2, b13, b2, top_k=cfg.k)(x, lg)), y_ref, None, "layer")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_decode_steps(fmt):
    """Three steps of two sequences: project, append, read the whole context."""
    g = synth.rng(330)
    heads, dim, H, page = 2, 64, 96, 4
    w = synth.to_bf16_bits(g.standard_normal((2 * heads * dim, H), dtype=np.float32) * np.float32(0.1))
    q, s, _ = mx.nvfp4_quantize(bf16_dev(w), 500.0, tiled=False)
    gs = (40.0, 60.0) if fmt == "nvfp4" else (1.0, 1.0)
    code = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}[fmt]
    c = mx.PagedCache(6, page, heads, dim, dim, code, *gs)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[4, 1], [0, 5]])
    have = [0, 2]
    want = [[], []]
    first = synth.to_bf16_bits(g.standard_normal((2, 2, heads * dim)))  # sequence 1's first two tokens
    c.write(*(bf16_dev(first[i].reshape(2, heads, dim)) for i in range(2)), table, i32([0, 0, 2]))
    want[1] += [(first[0][t], first[1][t]) for t in range(2)]
    for step in range(3):
        x = synth.to_bf16_bits(g.standard_normal((2, H), dtype=np.float32))
        kv = mx.fp4_matvec(bf16_dev(x), q, s, fmt=mx.FMT_NVFP4, global_scale=500.0)
        ref, mag = V.matvec_ref(x, q.cpu().numpy(), s.cpu().numpy(), None, 500.0)
        assert np.all(np.abs(bf16_host_f64(kv) - ref) <= 2.0 ** -8 * np.abs(ref) + 100 * 2.0 ** -24 * mag)
        k, v = (t.view(2, heads, dim) for t in kv.chunk(2, dim=1))
        c.write(k, v, table, i32([0, 1, 2]), i32(have))
        bits = bf16_host_bits(kv)
        for b in range(2):
            want[b].append(tuple(np.split(bits[b], 2)))
        have = [h + 1 for h in have]
        rows = sum(have)
        ko, vo = c.read(table, i32([0, have[0], rows]), rows=rows)
        for i, got in enumerate((ko, vo)):
            held = np.stack([t[i] for seq in want for t in seq]).reshape(rows, heads, dim)
            np.testing.assert_array_equal(bf16_host_bits(got), C.bf16_bits(C.decode_ref(*C.encode_ref(held, fmt, gs[i]), fmt, gs[i])))


def test_router_training_step_beside_the_layer():
    """One step of a router: the balance loss on the routing that the layer uses, its gradient in the router's weight
    by the chain rule."""
    g = synth.rng(331)
    T, H, E, k = 40, 64, 8, 2
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).cuda()
    w = torch.from_numpy((g.standard_normal((E, H)) * 0.2).astype(np.float32)).cuda().requires_grad_()
    logits = x @ w.t()
    ids, _, offs, _ = mx.route(logits.detach().contiguous(), k)
    loss, counts = mx.balance_loss(logits, ids)
    (0.02 * loss).backward()
    assert torch.equal(counts, offs[1:] - offs[:-1])
    l64 = logits.detach().cpu().numpy()
    ref, n, gl = B.balance_ref(l64, ids.cpu().numpy(), None, float(np.float32(0.02)))
    assert loss.item() == pytest.approx(ref, rel=200 * 2.0 ** -24)
    want = gl.T @ x.cpu().numpy().astype(np.float64)
    # each product off by the gradient's tolerance (dp <= 64 u here, D <= 8 / (2 * 1600) * 80), T of them in a sum
    tol = 0.02 * 2 * 0.2 * 128 * 2.0 ** -24 * np.abs(x.cpu().numpy()).sum(0)[None, :] + 42 * 2.0 ** -24 * (np.abs(gl).T @ np.abs(x.cpu().numpy()))
    assert np.all(np.abs(w.grad.cpu().numpy() - want) <= tol)
