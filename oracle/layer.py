"""Oracle of a layer's row-wise operators: the formulas of ``include/vf_relayout.h``
("Gated activation", "Root-mean-square norm") in float64 on CPU tensors, sharing
no code with the library."""
import torch


def sigmoid(g):
    """1 / (1 + exp(-g)) in float64, by the exponential that cannot overflow."""
    e = torch.exp(-g.abs())
    return torch.where(g >= 0, 1 / (1 + e), e / (1 + e))


def glu(gate, up):
    g, u = gate.double(), up.double()
    return g * sigmoid(g) * u


def glu_backward(grad, gate, up):
    d, g, u = grad.double(), gate.double(), up.double()
    s = sigmoid(g)
    return d * u * s * (1 + g * (1 - s)), d * g * s


def total(x, residual):
    """x + residual, rounded to the type by way of float32, as the header states."""
    return (x.float() + residual.float()).to(x.dtype)


def norm(h, weight, eps):
    h = h.double()
    r = 1 / torch.sqrt((h * h).sum(dim=1, keepdim=True) / h.shape[1] + eps)
    return h * r * weight.double()


def norm_backward(grad, h, weight, eps, grad_total=None):
    """(grad_x, grad_weight, scale of grad_x's terms, magnitudes of grad_weight's)."""
    h, g, w = h.double(), grad.double(), weight.double()
    M = h.shape[1]
    r = 1 / torch.sqrt((h * h).sum(dim=1, keepdim=True) / M + eps)
    dx = r * (w * g - h * r * r * (w * g * h).sum(dim=1, keepdim=True) / M)
    mag = r * ((w * g).abs() + h.abs() * r * r * (w * g * h).abs().sum(dim=1, keepdim=True) / M)
    if grad_total is not None:
        dx = dx + grad_total.double()
        mag = mag + grad_total.double().abs()
    terms = g * h * r
    return dx, terms.sum(dim=0), mag, terms.abs().sum(dim=0)
