"""Blocks on 8-bit checkpoints that share one scratch: what each of them keeps, and the same
bits as blocks with buffers of their own over a training step of three of them."""
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL
from grouped_gemm_moe_gb300 import layer as L
from grouped_gemm_moe_gb300 import workloads as W

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _scratch(cfg):
    return BL.BlockScratch(cfg.T, cfg.d, cfg.E, cfg.K, cfg.I, cfg.shared_I, dev())


def _tensors(obj):
    out = []
    for v in vars(obj).values():
        out += [t for t in (v if isinstance(v, (tuple, list)) else (v,)) if torch.is_tensor(t)]
    return out


@pytest.mark.parametrize("shared_I", [0, 384])
def test_what_a_block_keeps(shared_I):
    """Beside its gradients: the checkpoint, out and z, and less than a twentieth of those for
    indexes, router weights and statistics."""
    cfg = W.small_config("kept", T=2048, d=1024, E=8, K=4, I=384, R=1, shared_I=shared_I)
    inp = W.make_inputs(cfg)
    scratch = _scratch(cfg)
    weights = {k: v.to(dev()) for k, v in inp.items() if k.startswith("w")}
    gain = torch.ones(cfg.d, device=dev())
    blocks = [BL.MoEBlock(L.MoELayer(cfg.T, cfg.d, cfg.E, cfg.K, cfg.I, cfg.R, weights, cfg.renorm,
                                     dev(), ckpt8=True, scratch=scratch), gain, gain)
              for _ in range(2)]
    size = lambda ts: sum(n for n in {t.untyped_storage().data_ptr():  # noqa: E731
                                      t.untyped_storage().nbytes() for t in ts}.values())
    shared = {t.untyped_storage().data_ptr() for t in _tensors(scratch) + list(weights.values()) + [gain]}
    T, d, TK = cfg.T, cfg.d, cfg.T * cfg.K
    kept = (T * d + TK * 2 * cfg.I + TK * d + T * 2 * shared_I) * 34 // 32 + 2 * (2 * T * d)
    for block in blocks:
        grads = [t for n, t in vars(block.layer).items() if n.startswith(("dw_", "dws_"))]
        own = [t for t in _tensors(block) + _tensors(block.layer)
               if t.is_cuda and t.untyped_storage().data_ptr() not in shared]
        extra = size(own) - size(grads) - kept
        assert 0 <= extra <= kept // 20, (size(own), kept, extra)
        rows = {t.data_ptr() for t in own if t.dtype == BF and t.numel() >= T * d}
        assert rows == {block.out.data_ptr(), block.z.data_ptr()}
    assert blocks[0].out.data_ptr() != blocks[1].out.data_ptr()


def _step(blocks, routers, xs, dout):
    """A training step of a stack of blocks with their routers: every result, cloned as it
    comes."""
    res, x = [], xs
    for b, r in zip(blocks, routers):
        xn = b.norm(x)
        x = b.forward(xn.float() @ r)
        res.append(x.clone())
    for b, r in reversed(list(zip(blocks, routers))):
        dxn, dlogits = b.backward(dout)
        res += [b.xn.float().t() @ dlogits, dlogits.clone()]
        dxn += (dlogits @ r.t()).to(BF)
        dout = b.backward_norm(dxn)
        res += [dout.clone(), b.dgain_in.clone(), b.dgain_out.clone(), b.dgate.clone(),
                b.layer.dw_gate.clone(), b.layer.dw_down.clone()]
    return res


@pytest.mark.parametrize("shared_I", [0, 256])
def test_a_step_of_three_blocks(shared_I):
    cfg = W.small_config("stack", T=384, d=128, E=8, K=2, I=128, R=2, shared_I=shared_I)
    drawn = [W.make_inputs(cfg, seed=s, with_backward=True) for s in (1, 2, 3)]
    g = torch.Generator(device=dev()).manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
    routers = [rand(cfg.d, cfg.E) for _ in drawn]
    vecs = [(1 + 0.1 * rand(cfg.d), 1 + 0.1 * rand(cfg.d), 1 + 0.1 * rand(4, cfg.d)) for _ in drawn]
    x, dout = drawn[0]["x"].to(dev()), drawn[0]["dout"].to(dev())

    def blocks(scratch):
        return [BL.MoEBlock(L.layer_from_config(cfg, d, dev(), ckpt8=True, scratch=scratch), *v,
                            span=100, scale=0.5) for d, v in zip(drawn, vecs)]
    alone = _step(blocks(None), routers, x, dout)
    sharing = blocks(_scratch(cfg))
    for _ in range(2):      # a second step finds nothing of the first one's
        for got, want in zip(_step(sharing, routers, x, dout), alone):
            assert torch.equal(got, want)


def test_a_shared_xn_is_not_taken_for_anothers():
    cfg = W.small_config("order", T=64, d=128, E=8, K=2, I=128, R=2)
    inp = W.make_inputs(cfg, with_backward=True)
    gain, x = torch.ones(cfg.d, device=dev()), inp["x"].to(dev())
    scratch = _scratch(cfg)
    a, b = (BL.MoEBlock(L.layer_from_config(cfg, inp, dev(), ckpt8=True, scratch=scratch), gain)
            for _ in range(2))
    a.norm(x)
    b.norm(x)
    with pytest.raises(RuntimeError):
        a.forward(inp["logits"].to(dev()))
    b.forward(inp["logits"].to(dev()))


def test_a_layer_in_a_block_still_runs_alone():
    cfg = W.small_config("alone", T=64, d=128, E=8, K=2, I=128, R=2)
    inp = W.make_inputs(cfg)
    logits, x = inp["logits"].to(dev()), inp["x"].to(dev())
    want = L.layer_from_config(cfg, inp, dev()).forward(logits, x)
    layer = L.layer_from_config(cfg, inp, dev())
    BL.MoEBlock(layer, torch.ones(cfg.d, device=dev()))
    got = layer.forward(logits, x)
    assert torch.equal(got, want) and layer.forward(logits, x).data_ptr() == got.data_ptr()


@pytest.mark.parametrize("T,d", [(1, 8), (5003, 2056), (700, 8200), (30001, 136)])
def test_norm_in_backward_over_the_residuals_gradient(T, d):
    """dx over dres gives the bits of a dx of its own."""
    g = torch.Generator(device=dev()).manual_seed(T)
    dxn, x, dres = (torch.randn(T, d, generator=g, device=dev()).to(BF) for _ in range(3))
    gain, rstd = torch.rand(d, generator=g, device=dev()), torch.rand(T, generator=g, device=dev())
    want, dgain = B.moe_norm_in_backward(dxn, x, gain, rstd, dres)
    got, dgain2 = B.moe_norm_in_backward(dxn, x, gain, rstd, dres, out=(dres, torch.empty_like(gain)))
    assert got.data_ptr() == dres.data_ptr()
    assert torch.equal(got, want) and torch.equal(dgain, dgain2)
