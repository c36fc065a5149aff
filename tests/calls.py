"""Every call of the binding that takes a stream, on small inputs: name -> a function of keyword
arguments (stream=) that returns the call's tensors by name. Shared by the stream tests."""

import torch

import token_weight_scans_b200 as tw
from tests import delta_ref as ref


def all_calls(device, B=2, H=2, T=70, d=32, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(device)  # noqa: E731
    x, gg, v, dy = r(B, H, T, d), r(B, H, T, d), r(B, H, T, d), r(B, H, T, d)
    eta, alpha = 0.01 * torch.sigmoid(r(B, H, T)), torch.sigmoid(r(B, H, T) + 4)
    W0, S, hid = 0.1 * r(H, d, d), 0.1 * r(B, H, d, d), r(B, H, T, d)
    dl = {n: t.to(device) for n, t in ref.draw(B, H, H, T, d, d, "f32", True, seed=seed).items()}
    rule = [dl[n] for n in ("q", "k", "v", "beta", "log_alpha")]
    rows, w = r(B, T, H, d), 1 + 0.1 * r(d)
    pool = dl["S0"].clone()

    state = S.clone()

    def reset(to, like, stream=None):  # the states as they were, on the call's stream
        if stream is None:
            return to.copy_(like)
        with torch.cuda.stream(stream):
            return to.copy_(like)

    def step(**kw):
        return dict(y=tw.gradlev_delta_step(*rule, reset(pool, dl["S0"], **kw), **kw))

    def decode(**kw):
        y, gt = tw.gradlev_decode_step(x, v, eta, alpha, W0, reset(state, S, **kw), **kw)
        return dict(y=y, g=gt)

    pair = lambda y, S: dict(y=y, S=S)  # noqa: E731
    return {
        "gradlev_scan_fwd": lambda **kw: dict(y=tw.gradlev_scan_fwd(x, gg, eta, alpha, W0, **kw)),
        "gradlev_scan_bwd": lambda **kw: tw.gradlev_scan_bwd(x, gg, eta, alpha, W0, dy, **kw),
        "gradlev_scan_fwd_state": lambda **kw: pair(
            *tw.gradlev_scan_fwd_state(x, gg, eta, alpha, W0, S, **kw)),
        "gradlev_scan_bwd_state": lambda **kw: tw.gradlev_scan_bwd_state(
            x, gg, eta, alpha, W0, dy, S, **kw),
        "gradlev_decode_step": decode,
        "gradlev_consistency_step": lambda **kw: tw.gradlev_consistency_step(
            x, gg, eta, alpha, W0, v, **kw),
        "gradlev_mlp2_recon": lambda **kw: tw.gradlev_mlp2_recon(
            x, hid, gg, v, eta, alpha, W0, W0, **kw),
        "gradlev_delta_fwd": lambda **kw: pair(*tw.gradlev_delta_fwd(*rule, dl["S0"], **kw)),
        "gradlev_delta_bwd": lambda **kw: tw.gradlev_delta_bwd(*rule, dl["dy"], dl["S0"], **kw),
        "gradlev_delta_step": step,
        "gradlev_qk_norm_rope_fwd": lambda **kw: pair(
            *tw.gradlev_qk_norm_rope_fwd(rows, rows, w, w, **kw)),
        "gradlev_qk_norm_rope_bwd": lambda **kw: tw.gradlev_qk_norm_rope_bwd(
            dy, dy, rows, rows, w, w, **kw),
    }


NAMES = sorted(all_calls("cpu"))
