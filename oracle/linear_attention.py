"""fp64 restatement of linear attention with a decay for each head, token by
token, with its gradients. Shapes: q, k [T,H,Dk], v [T,H,Dv], log_decay [H],
states [H,Dk,Dv] (one sequence; callers loop over sequences)."""
import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def forward(q, k, v, log_decay, h0=None):
    """S_t = gamma S_{t-1} + k_t v_t^T, o_t = S_t^T q_t: (o, S_{T-1})."""
    q, k, v, ld = (_f64(x) for x in (q, k, v, log_decay))
    T, H, Dk = q.shape
    S = np.zeros((H, Dk, v.shape[-1])) if h0 is None else _f64(h0).copy()
    gamma = np.exp(ld)[:, None, None]
    o = np.zeros((T, H, v.shape[-1]))
    for t in range(T):
        S = gamma * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = (S * q[t][:, :, None]).sum(1)
    return o, S


def backward(q, k, v, log_decay, h0, d_o, dh_final=None):
    """Reverse-mode gradients of <d_o, o> + <dh_final, S_{T-1}>: the chain rule
    applied to each token's update and readout, from the last to the first.
    Returns dq, dk, dv, dh0."""
    q, k, v, ld, d_o = (_f64(x) for x in (q, k, v, log_decay, d_o))
    T, H, Dk = q.shape
    Dv = v.shape[-1]
    gamma = np.exp(ld)[:, None, None]
    S = np.zeros((H, Dk, Dv)) if h0 is None else _f64(h0).copy()
    dq = np.zeros_like(q)
    for t in range(T):
        S = gamma * S + k[t][:, :, None] * v[t][:, None, :]
        dq[t] = (S * d_o[t][:, None, :]).sum(2)
    dS = np.zeros((H, Dk, Dv)) if dh_final is None else _f64(dh_final).copy()
    dk, dv = np.zeros_like(k), np.zeros_like(v)
    for t in reversed(range(T)):
        dS = dS + q[t][:, :, None] * d_o[t][:, None, :]     # the readout
        dk[t] = (dS * v[t][:, None, :]).sum(2)               # the update
        dv[t] = (dS * k[t][:, :, None]).sum(1)
        dS = gamma * dS
    return dq, dk, dv, dS


def magnitudes(q, k, v, log_decay, h0=None):
    """The recurrence of the absolute values: what rounding errors of the
    terms are proportional to. Returns (o, S) of |q|, |k|, |v|, |h0|."""
    a = [np.abs(_f64(x)) for x in (q, k, v)]
    return forward(*a, log_decay, None if h0 is None else np.abs(_f64(h0)))
