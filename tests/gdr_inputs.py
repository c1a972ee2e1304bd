"""Seeded inputs of the gated delta rule tests."""
import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(B, T, Hk, H, K, V, seed=0, dtype="bf16", state=True, decay=1.0, key_norm=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return {"q": unit(n(B, T, Hk, K)).to(DT[dtype]), "k": (key_norm * unit(n(B, T, Hk, K))).to(DT[dtype]),
            "v": n(B, T, H, V).to(DT[dtype]),
            "g": -decay * torch.nn.functional.softplus(n(B, T, H) - 2.0),
            "beta": torch.sigmoid(n(B, T, H)), "state": 0.3 * n(B, H, K, V) if state else None}


NAMES = ("q", "k", "v", "g", "beta")


def on_gpu(inp):
    return {n: None if x is None else x.cuda() for n, x in inp.items()}
