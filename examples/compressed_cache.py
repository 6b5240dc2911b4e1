"""Decode steps over a paged key/value cache, and the same after K-Means has compressed the older slots.

A request's old keys are clustered for each head (`km.fit_batched`), its values averaged over the same clusters
(`km.update`), and the centroids take the place of the tokens, each with the logarithm of its cluster's size as its
weight: softmax(q k + log n) counts a centroid as n equal keys.  Newer tokens stay exact.  Every step makes its tables
on the GPU, appends the new keys and values (normed and rotated) and attends over what the cache holds.

    python examples/compressed_cache.py --context 8192 --clusters 512
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import means_clustering_amd as km  # noqa: E402
from means_clustering_amd import kvcache  # noqa: E402


class Server:
    """One layer's cache and its requests, one of which decodes."""

    def __init__(self, q_heads, heads, dim, page_size, pages, max_pos, dtype=torch.bfloat16, device="cuda:0"):
        self.q_heads, self.heads, self.dim, self.page_size = q_heads, heads, dim, page_size
        self.k = torch.zeros(pages, page_size, heads, dim, dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.log_weight = torch.zeros(pages, heads, page_size, device=device)  # 0: a token
        self.free = torch.arange(pages, dtype=torch.int32, device=device)
        self.table = torch.full((1, pages), -1, dtype=torch.int32, device=device)
        self.held = torch.zeros(1, dtype=torch.int32, device=device)    # slots in the cache
        self.offset = torch.zeros(1, dtype=torch.int32, device=device)  # tokens seen but not held
        self.centroids = 0  # leading slots that hold centroids
        angle = torch.arange(max_pos, device=device)[:, None] * torch.pow(
            10000.0, -torch.arange(0, dim, 2, device=device) / dim)[None]
        self.rope = torch.cat([angle.cos(), angle.sin()], dim=1)
        self.norm = torch.ones(dim, device=device)
        self.ws = kvcache.Workspace(device)

    def step(self, qkv, rotate=True):
        """Appends the tokens of a packed projection [n, q_heads + 2 heads, dim] and returns their attention."""
        n, hq, h = qkv.shape[0], self.q_heads, self.heads
        new = torch.full_like(self.held, n)
        t = kvcache.tables(self.held, new, self.table, self.free, self.page_size, n, pos_offset=self.offset)
        turn = dict(positions=t.positions, rope=self.rope, q_weight=self.norm, k_weight=self.norm) if rotate else {}
        q = kvcache.append(qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:], self.k, self.v, t.slots, **turn)
        out = kvcache.attend(q, self.k, self.v, self.table, t.query_start, t.seq_lens, log_weight=self.log_weight,
                             max_new=n, ws=self.ws)
        self.free = self.free[int(t.page_start[-1]):]  # (a scheduler on the host knows this number by itself)
        self.held = t.seq_lens
        return out

    def compress(self, slots, clusters, iters=8):
        """Replaces the request's oldest `slots` tokens (whole pages) by `clusters` centroids (whole pages).

        The centroids of earlier calls stay as they are: K-Means would count each of them as one key.
        """
        p, h, d = self.page_size, self.heads, self.dim
        if slots % p or clusters % p or not 0 < clusters <= slots:
            raise ValueError("slots and clusters must be whole pages, and not more clusters than slots")
        first, last = self.centroids // p, (self.centroids + slots) // p
        if last * p > int(self.held):
            raise ValueError(f"the cache holds {int(self.held) - self.centroids} tokens, fewer than {slots}")
        old = self.table[0, first:last].clone()
        keys = self.k[old.long()].view(slots, h, d).transpose(0, 1).contiguous()
        values = self.v[old.long()].view(slots, h, d).transpose(0, 1).reshape(h * slots, d)
        # centroids start at keys spread over the context
        spread = keys[:, torch.arange(clusters, device=keys.device) * slots // clusters].float().contiguous()
        centroids, assign, counts, _ = km.fit_batched(keys, spread, iters)
        cluster = assign + torch.arange(h, dtype=torch.int32, device=keys.device)[:, None] * clusters
        means, _ = km.update(values, cluster.view(-1), torch.zeros(h * clusters, d, device=keys.device))
        # the centroids go into the first of the old pages, the others (whose weights are a token's, 0) are free again
        kept = old[:clusters // p]
        at = torch.arange(clusters, dtype=torch.int32, device=keys.device)
        kvcache.append(None, centroids.transpose(0, 1).to(keys.dtype).contiguous(),
                       means.view(h, clusters, d).transpose(0, 1).to(keys.dtype).contiguous(), self.k, self.v,
                       kept[(at // p).long()] * p + at % p)
        # (-inf where a cluster is empty)
        self.log_weight[kept.long()] = counts.view(h, clusters // p, p).transpose(0, 1).float().log()
        self.free = torch.cat([old[clusters // p:], self.free])
        self.table = torch.cat([self.table[0, :first], kept, self.table[0, last:],
                                old.new_full(((slots - clusters) // p,), -1)])[None]
        self.centroids += clusters
        self.held = self.held - (slots - clusters)
        self.offset = self.offset + (slots - clusters)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--context", type=int, default=8192, help="tokens of the prompt")
    ap.add_argument("--clusters", type=int, default=512, help="centroids that replace all but the last 512 tokens")
    ap.add_argument("--topics", type=int, default=256, help="directions that the prompt's keys and values scatter around")
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--rotate", action="store_true", help="norm and rotate queries and keys (equal keys at different "
                    "positions then differ, and take more clusters)")
    a = ap.parse_args()
    hq, h, d, p = 32, 8, 128, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    topic = torch.randn(a.topics, h, d, generator=g, device="cuda")
    pick = torch.randint(a.topics, (a.context,), generator=g, device="cuda")
    qkv = torch.randn(a.context + a.steps, hq + 2 * h, d, generator=g, device="cuda")
    qkv[:a.context, hq:] = topic[pick].repeat(1, 2, 1) + 0.2 * qkv[:a.context, hq:]
    qkv = qkv.to(torch.bfloat16)
    servers = [Server(hq, h, d, p, (a.context + a.steps) // p + 2, a.context + a.steps) for _ in range(2)]
    for s in servers:
        s.step(qkv[:a.context], a.rotate)
    old = (a.context - 512) // p * p
    servers[1].compress(old, a.clusters)
    print(f"{a.context} tokens: {int(servers[0].held)} slots exact, {int(servers[1].held)} compressed")
    for i in range(a.steps):
        exact, short = (s.step(qkv[a.context + i:a.context + i + 1], a.rotate).float() for s in servers)
        print(f"step {i}: relative difference {float((exact - short).norm() / exact.norm()):.4f}")


if __name__ == "__main__":
    main()
