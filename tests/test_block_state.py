"""What LatentMoEBlock keeps from call to call, on the host: its forward call is replaced by nothing, its tensors
are in host memory (the router methods then end at the library's check for CUDA tensors)."""
import weakref

import pytest
import torch

D, L, E, I, K = 256, 128, 8, 128, 2


@pytest.fixture(scope="module")
def lm():
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


@pytest.fixture
def blk(lm, monkeypatch):
    monkeypatch.setattr(lm, "latent_moe_forward", lambda *a, **k: None)
    z = torch.zeros
    return lm.LatentMoEBlock(z(E, D), z(L, D), z(L), z(E, I, L), z(E, I, L), z(E, L, I), z(E, L), z(D, L), z(D), z(D), K)


def x(T, dtype=torch.bfloat16):
    return torch.zeros(T, D, dtype=dtype)


def refused(fn, cfg):
    with pytest.raises(ValueError, match="forward call"):
        fn(cfg)


def taken(fn, cfg):
    with pytest.raises(ValueError, match="CUDA tensor"):   # past the block's own check
        fn(cfg)


def test_routing_of_a_call_that_did_not_run_is_refused(blk):
    # a smaller call than the last has its logits elsewhere in the workspace
    blk.forward(x(300))
    for fn in (blk.router_losses, blk.router_grad):
        for T in (40, 299, 301, 3000):
            refused(fn, blk.config(T))
        taken(fn, blk.config(300))
        taken(fn, blk.config(300, "f32", "bf16"))   # the types of x and out do not matter
    blk.forward(x(40, torch.float32))
    taken(blk.router_losses, blk.config(40))
    refused(blk.router_losses, blk.config(300))


def test_routing_of_another_block_is_refused(lm, blk):
    blk.forward(x(40))
    c = blk.config(40)
    for change in (dict(d_model=512), dict(n_experts=16), dict(top_k=1), dict(d_latent=256), dict(d_ff=256)):
        refused(blk.router_losses, lm.Config(**{**c.__dict__, **change}))


def test_routing_after_a_call_that_failed_is_refused(lm, blk, monkeypatch):
    blk.forward(x(40))

    def fails(*a, **k):
        raise lm.LmoeError(-5, "latent_moe_forward")
    monkeypatch.setattr(lm, "latent_moe_forward", fails)
    with pytest.raises(lm.LmoeError):
        blk.forward(x(40))
    refused(blk.router_losses, blk.config(40))


def test_routing_after_a_larger_workspace_is_refused(blk):
    blk.forward(x(40))
    blk.workspace(blk.config(4000))       # a new one: nothing has run in it
    refused(blk.router_losses, blk.config(40))


def test_workspace_of_a_captured_call_is_kept(blk, monkeypatch):
    capturing = [False]
    monkeypatch.setattr(blk, "_capturing", lambda: capturing[0], raising=False)
    blk.forward(x(40))
    blk.forward(x(400))                      # the first one was in no graph: gone
    assert not getattr(blk, "_kept", [])
    capturing[0] = True
    blk.forward(x(40))
    capturing[0] = False
    used = weakref.ref(blk._ws)
    blk.forward(x(4000))
    assert used() is not None and used() is not blk._ws
    # the router methods' views count as well
    blk.forward(x(4000))
    capturing[0] = True
    taken(blk.router_losses, blk.config(4000))
    capturing[0] = False
    again = weakref.ref(blk._ws)
    blk.forward(x(6000))
    assert again() is not None and used() is not None


def test_workspace_made_by_a_captured_call_is_its_own(blk, monkeypatch):
    # zeroed only when the graph runs: an eager call takes another
    capturing = [True]
    monkeypatch.setattr(blk, "_capturing", lambda: capturing[0], raising=False)
    blk.forward(x(40))
    first = weakref.ref(blk._ws)
    blk.forward(x(40))                       # (the same capture goes on with it)
    assert blk._ws is first()
    capturing[0] = False
    blk.forward(x(40))
    assert blk._ws is not first() and first() is not None


def test_views_are_the_layouts(lm, blk):
    blk.forward(x(40))
    cfg = blk.config(40)
    lay = lm.lmoe_get_workspace_layout(cfg)
    logits, idx = blk._routing(cfg)
    assert logits.shape == (40, E) and idx.shape == (40, K)
    assert logits.data_ptr() - blk._ws.data_ptr() == lay["logits"] and idx.data_ptr() - blk._ws.data_ptr() == lay["topk_idx"]
    logits, idx = blk._routing(blk.config(0))
    assert logits.shape == (0, E) and idx.shape == (0, K)
