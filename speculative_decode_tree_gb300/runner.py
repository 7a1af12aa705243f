"""Device buffers for one verify batch, driven through the C ABI.

Holds the inputs on the GPU, the plan, the caller-owned workspace and the
outputs, and calls the batched entry point.  Plumbing only: all compute runs
in the library's kernels.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B
from .workloads import VerifyInputs


class DeviceVerify:
    def __init__(self, inp: VerifyInputs, device: str = "cuda", kernel: Optional[int] = None,
                 check_pool: bool = True, plan: Optional[B.Plan] = None):
        dev = torch.device(device)
        self.inp = inp
        self.kv_pool = inp.kv_pool.to(dev)
        self.kv_indices = inp.kv_indices.to(dev)
        self.kv_indptr = inp.kv_indptr.to(dev)
        self.prefix_lens = inp.prefix_lens.to(dev)
        self.tree_parent = inp.tree_parent.to(dev).contiguous()
        self.q_latent = inp.q_latent.to(dev)
        self.q_rope = inp.q_rope.to(dev)
        pool_rows = inp.pool_rows if check_pool else 0
        if plan is not None:
            self.plan = plan
        elif kernel is None:
            self.plan = B.ddtree_verify_mla_plan(inp.batch, inp.n_nodes, inp.n_heads,
                                                 inp.prefix_lens.tolist(), pool_rows)
        else:
            self.plan = B.ddtree_verify_mla_plan_ex(inp.batch, inp.n_nodes, inp.n_heads,
                                                    inp.prefix_lens.tolist(), pool_rows, 0, kernel)
        rows = inp.batch * inp.n_nodes
        self.out = torch.empty(rows, inp.n_heads, 512, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(rows, inp.n_heads, dtype=torch.float32, device=dev)
        self.workspace = torch.empty(B.ddtree_verify_mla_workspace_size(self.plan),
                                     dtype=torch.uint8, device=dev)

    def run(self, stream=None) -> None:
        B.ddtree_verify_mla_batched(self.plan, self.q_latent, self.q_rope, self.kv_pool,
                                    self.kv_indices, self.kv_indptr, self.prefix_lens,
                                    self.tree_parent, self.inp.sm_scale, self.out, self.lse,
                                    self.workspace, stream)

    def run_timed(self, stage_events, stream=None) -> None:
        B.ddtree_verify_mla_batched_timed(self.plan, self.q_latent, self.q_rope, self.kv_pool,
                                          self.kv_indices, self.kv_indptr, self.prefix_lens,
                                          self.tree_parent, self.inp.sm_scale, self.out, self.lse,
                                          self.workspace, stage_events, stream)

    def run_single(self, stream=None) -> None:
        """The single-request entry point (batch 1)."""
        assert self.inp.batch == 1
        B.ddtree_verify_mla(self.q_latent, self.q_rope, self.kv_pool, self.kv_indices,
                            int(self.inp.prefix_lens[0]), self.tree_parent, self.inp.n_nodes,
                            self.inp.n_heads, self.inp.sm_scale, self.out, self.lse,
                            self.workspace, stream)

    def status(self, stream=None) -> int:
        return B.ddtree_verify_mla_check(self.workspace, stream)


class DeviceAccept:
    """Device copies of an acceptance workload and its output buffers."""

    def __init__(self, inp, device: str = "cuda"):
        dev = torch.device(device)
        self.inp = inp
        self.logits = inp.logits.to(dev).contiguous()
        self.draft = inp.draft_tokens.to(dev).contiguous()
        self.parent = inp.tree_parent.to(dev).contiguous()
        self.kv_indices = inp.kv_indices.to(dev)
        self.kv_indptr = inp.kv_indptr.to(dev)
        self.prefix_lens = inp.prefix_lens.to(dev)
        nb, nt = inp.batch, inp.n_nodes
        i32 = torch.int32
        self.accept_len = torch.empty(nb, dtype=i32, device=dev)
        self.next_token = torch.empty(nb, dtype=i32, device=dev)
        self.accepted_nodes = torch.empty(nb, nt, dtype=i32, device=dev)
        self.commit_indices = torch.empty(nb, nt, dtype=i32, device=dev)
        self.freed_indices = torch.empty(nb, nt, dtype=i32, device=dev)
        self.workspace = torch.empty(B.ddtree_accept_greedy_workspace_size(nb, nt), dtype=torch.uint8,
                                     device=dev)

    def run(self, stream=None) -> None:
        B.ddtree_accept_greedy(self.logits, self.draft, self.parent, self.kv_indices, self.kv_indptr,
                               self.prefix_lens, self.accept_len, self.next_token, self.accepted_nodes,
                               self.commit_indices, self.freed_indices, self.workspace, stream)

    def status(self, stream=None) -> int:
        return B.ddtree_verify_mla_check(self.workspace, stream)

    def outputs(self) -> dict:
        return {"accept_len": self.accept_len.cpu().numpy(), "next_token": self.next_token.cpu().numpy(),
                "accepted_nodes": self.accepted_nodes.cpu().numpy(),
                "commit_indices": self.commit_indices.cpu().numpy(),
                "freed_indices": self.freed_indices.cpu().numpy()}



class DeviceStep:
    """Static buffers of one decode step of the target model around verify
    attention, each call marshalled once: step maps (page growth, index layout,
    slots, positions), latent append (pool rows, rotated queries), verify.

    The caller fills `prefix_lens`, `tree_parent`, `pages_held`, `free_head`,
    `kv_new` [B*T, 576], `q` [B*T, H, 576] (latent part as absorbed, rope part
    not yet rotated) and calls `run`; `out` and `lse` are the verify outputs and
    `pages_held_out`, `free_head_out` what the step took.  `run` can be captured
    into a graph and replayed with other contents up to `max_prefix`."""

    def __init__(self, batch: int, n_nodes: int, n_heads: int, max_prefix: int, page_size: int, kv_pool: torch.Tensor,
                 page_table: torch.Tensor, free_pages: torch.Tensor, rope: B.Rope, sm_scale: float,
                 latent_weight: Optional[torch.Tensor] = None):
        dev, i32, bf = kv_pool.device, torch.int32, torch.bfloat16
        n_pages, n = int(kv_pool.shape[0]) // page_size, batch * n_nodes

        def ints(*shape):
            return torch.zeros(*shape, dtype=i32, device=dev)
        self.prefix_lens, self.tree_parent = ints(batch), ints(batch, n_nodes)
        self.pages_held, self.free_head = ints(batch), ints(1)
        self.pages_held_out, self.free_head_out = ints(batch), ints(1)
        self.kv_indptr, self.kv_indices = ints(batch + 1), ints(batch * (max_prefix + n_nodes))
        self.new_slots, self.positions, self.status_word = ints(n), ints(n), ints(1)
        self.kv_new = torch.zeros(n, 576, dtype=bf, device=dev)
        self.q = torch.zeros(n, n_heads, 576, dtype=bf, device=dev)
        self.out = torch.empty(n, n_heads, 512, dtype=bf, device=dev)
        self.lse = torch.empty(n, n_heads, dtype=torch.float32, device=dev)
        self.plan = B.ddtree_verify_mla_plan(batch, n_nodes, n_heads, [max_prefix] * batch, int(kv_pool.shape[0]))
        self.plan.q_latent_row_stride = self.plan.q_rope_row_stride = 576
        self.workspace = torch.empty(B.ddtree_verify_mla_workspace_size(self.plan), dtype=torch.uint8, device=dev)
        q_rope = self.q[..., 512:]
        self._calls = (
            B.BoundStepMaps(page_table, self.prefix_lens, n_nodes, page_size, n_pages, self.kv_indptr, self.kv_indices,
                            self.new_slots, self.positions, tree_parent=self.tree_parent, pages_held=self.pages_held,
                            free_pages=free_pages, free_head=self.free_head, pages_held_out=self.pages_held_out,
                            free_head_out=self.free_head_out, status=self.status_word),
            B.BoundMlaAppend(rope, self.kv_new, self.positions, self.new_slots, kv_pool, latent_weight=latent_weight,
                             q_rope=q_rope, q_out=q_rope, status=self.status_word),
            B.BoundVerify(self.plan, self.q[..., :512], q_rope, kv_pool, self.kv_indices, self.kv_indptr,
                          self.prefix_lens, self.tree_parent, sm_scale, self.out, self.lse, self.workspace))

    def run(self, stream=None) -> None:
        for call in self._calls:
            call(stream)

    def status(self, stream=None) -> int:
        """Status bits of the last run, which `stream` was given to (synchronises); clears those
        of the maps and the append.  The clear is over when this returns, so a run that
        follows, on whatever stream, keeps its bits."""
        bits = B.ddtree_verify_mla_check(self.workspace, stream) | int(self.status_word)
        self.status_word.zero_()
        torch.cuda.current_stream(self.status_word.device).synchronize()
        return bits
