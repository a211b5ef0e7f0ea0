"""Plain 64-bit forms of the operators of experts and of dropout, from numpy and torch indexing."""
import numpy as np
import torch


def sort_reference(ids, experts):
    """(position, offsets) of a stable sort of the valid ids, by numpy."""
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    pairs = np.nonzero((flat >= 0) & (flat < experts))[0]
    pairs = pairs[np.argsort(flat[pairs], kind="stable")]
    position = np.full(flat.shape, -1, dtype=np.int32)
    position[pairs] = np.arange(len(pairs))
    offsets = np.searchsorted(flat[pairs], np.arange(experts + 1)).astype(np.int32)
    return torch.from_numpy(position.reshape(ids.shape)), torch.from_numpy(offsets)


def make_ids(tokens, k, experts, seed, none=0.0, dtype=torch.int64, device="cuda"):
    """Distinct experts for every token, some more in demand; a share `none` of the pairs without."""
    gen = torch.Generator(device=device).manual_seed(seed)
    demand = torch.randn(experts, generator=gen, device=device)
    logits = torch.randn(tokens, experts, generator=gen, device=device) + demand
    ids = logits.topk(min(k, experts), 1).indices
    if k > experts:
        ids = torch.cat([ids] * (k // experts + 1), 1)[:, :k].contiguous()
    if none:
        ids[torch.rand(tokens, k, generator=gen, device=device) < none] = -1
    return ids.to(dtype)


def philox(c0, c1, offset, seed):
    """Philox4x32-10 at the counters (c0, c1, offset) under `seed`, in unsigned 64-bit numpy."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    x0, x1 = np.broadcast_arrays(np.asarray(c0, dtype=u), np.asarray(c1, dtype=u))
    x = [x0, x1, np.full_like(x0, offset & 0xFFFFFFFF), np.full_like(x0, (offset >> 32) & 0xFFFFFFFF)]
    for i in range(10):
        k0 = u(((seed & 0xFFFFFFFF) + i * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = u((((seed >> 32) & 0xFFFFFFFF) + i * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(b >> u(32)) ^ x[1] ^ k0, b & low, (a >> u(32)) ^ x[3] ^ k1, a & low]
    return x


def kept(rows, n, p, seed, offset):
    """(mask, scale) of dropout, by numpy."""
    block, row = np.arange(-(-n // 8)), np.arange(rows)
    words = philox(block[None, :], row[:, None], offset, seed)
    numbers = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 2)
    q = int(np.floor(p * 65536 + 0.5))
    return torch.from_numpy(numbers.reshape(rows, -1)[:, :n] >= np.uint64(q)), 65536.0 / (65536 - q)
