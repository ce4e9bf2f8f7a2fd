"""What automatic differentiation is told: derivatives that the losses do not have are refused, and tensors that
they overwrite count as modified."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from quantized_optimizer_state_gb300 import fo, losses

CALLS = {
    "token_logprobs": lambda x: losses.token_logprobs(x, torch.zeros(3, dtype=torch.long, device=x.device), top_k=2),
    "distill_loss": lambda x: losses.distill_loss(x, torch.zeros(3, 2, dtype=torch.int32, device=x.device), torch.zeros(3, 2, device=x.device)),
    "distill_loss_grad": lambda x: losses.distill_loss_grad(x, torch.zeros(3, 2, dtype=torch.int32, device=x.device),
                                                            torch.zeros(3, 2, device=x.device)),
}


def refused(call, device):
    x, tangent = torch.randn(3, 10, device=device), torch.ones(3, 10, device=device)
    with forward_ad.dual_level():
        for leaf in (x, x.clone().requires_grad_(True)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call(forward_ad.make_dual(leaf, tangent))
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                call(forward_ad.make_dual(leaf, tangent))
    return x


@pytest.mark.parametrize("name", CALLS)
def test_forward_mode_is_refused(name):
    refused(CALLS[name], "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_forward_mode_is_refused_on_the_gpu(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = refused(CALLS[name], "cuda")
    CALLS[name](x)                            # no level is open any more
    with forward_ad.dual_level():
        CALLS[name](x)                        # and without a tangent there is nothing to lose


@pytest.mark.gpu
def test_a_gradient_in_the_logits_place_counts_as_a_change():
    """A graph that keeps the logits for its own backward pass says so instead of reading the gradient as logits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ids, y = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    stats, one = torch.empty(3, fo.FO_LOSS_STATS, device="cuda"), torch.ones(3, device="cuda")
    tokens = torch.zeros(3, dtype=torch.long, device="cuda")

    def wrapped(z):
        losses.distill_loss_grad(z, ids, y, out=z)

    def fused(z):
        fo.fo_distill(z, ids, y, grad=z)

    def apart(z):
        fo.fo_distill(z, ids, y, stats=stats)
        fo.fo_distill_grad(z, ids, y, stats, one, z)

    def logprobs(z):
        fo.fo_token_logprobs(z, stats=stats)
        fo.fo_token_logprobs_grad(z, stats, z, tokens, one)

    for overwrite in (wrapped, fused, apart, logprobs):
        h = torch.randn(3, 10, device="cuda", requires_grad=True)
        for use in (lambda x: x.logsumexp(1), lambda x: losses.token_logprobs(x, tokens).logp, lambda x: losses.distill_loss(x, ids, y)):
            x = h * 2
            out = use(x)
            overwrite(x.detach())
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                out.sum().backward()
    with torch.inference_mode():              # such tensors keep no count
        x = torch.randn(3, 10, device="cuda")
        losses.distill_loss_grad(x, ids, y, out=x)
