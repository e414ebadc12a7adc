"""Device state of a batch of sequences decoding with Token Recycling.

`TRState` owns the tensors one decoding loop needs (the adjacency matrices,
the loop state, the KV cache of the verification layer, the per-step outputs
and the workspaces) and calls the libtr ABI on the current stream.  It does
no arithmetic itself.  A step is

    state.verify(Q, Kt, Vt)          # tree attention for the current tree
    ... the target produces logits (or hidden states) for state.tree_tok ...
    state.finish(logits=...)         # top-K, accept, update, KV commit, next tree

or, without a draft (one token per sequence, the root's),

    state.decode(Q, Kn, Vn)          # append the root's K/V, attention of one token
    state.finish_decode(logits)      # top-K, update of the root's row, next root and tree

and the two may alternate (``single_token=True``).  With ``budget`` the attention weights that the
cached rows gather in decode are kept, and evict() cuts every sequence longer
than the budget down to it.  L then no longer is a token's position.

With ``rope`` (a Rope) the state norms and rotates queries and keys itself and keeps
count of the positions (``pos``, the roots').  Its rows come straight from the projection:

    state.verify(*state.rotate(Q, K, V))       # the tree's rows, at pos + depth
    ... state.finish(logits=..., Kt=state.Kt, Vt=state.Vt) ...
    state.decode(Q, Kn, Vn)                    # the roots' rows, at pos

Every call is asynchronous and allocation-free after construction, so whole
loops can be captured in a CUDA graph.
"""
from __future__ import annotations

import torch

from . import (TR_INIT_INHERIT, TR_UPD_ALL, KVCache, Rope, Tree, make_step_args, tr_accept, tr_decode_attn,
               tr_decode_attn_workspace_bytes, tr_get_status, tr_init_matrix, tr_kv_append, tr_kv_append_rope,
               tr_kv_append_workspace_bytes, tr_kv_evict, tr_kv_evict_workspace_bytes, tr_qkv_rope, tr_retrieve,
               tr_sample, tr_step, tr_step_sampled, tr_step_workspace_bytes, tr_topk, tr_topk_workspace_bytes, tr_update,
               tr_verify_attn, tr_verify_attn_workspace_bytes, workspace)


class TRState:
    def __init__(self, tree: Tree, B: int, V: int, m_dtype=torch.int64, Hq=0, Hkv=0, d=128, cap=0,
                 logits_dtype=torch.float32, D=0, device="cuda", single_token=False, budget=0, recent=0,
                 rope: Rope | None = None):
        self.tree = tree
        self.B, self.V, self.K, self.N = B, V, tree.K, tree.N
        self.Dmax = tree.max_depth
        self.device = device
        self.logits_dtype = logits_dtype
        self.D = D
        dev = dict(device=device)
        self.M = torch.zeros(B, V, tree.K, dtype=m_dtype, **dev)
        self.root = torch.zeros(B, dtype=torch.int32, **dev)
        self.L = torch.zeros(B, dtype=torch.int32, **dev)
        self.tree_tok = torch.zeros(B, self.N, dtype=torch.int32, **dev)
        self.ids = torch.zeros(B * self.N, tree.K, dtype=torch.int32, **dev)
        self.vals = torch.zeros(B * self.N, tree.K, dtype=torch.float32, **dev)
        self.acc_len = torch.zeros(B, dtype=torch.int32, **dev)
        self.path = torch.zeros(B, self.Dmax + 1, dtype=torch.int32, **dev)
        self.committed = torch.zeros(B, self.Dmax + 1, dtype=torch.int32, **dev)
        self.attention = Hq > 0
        if self.attention:
            self.Hq, self.Hkv, self.d, self.cap = Hq, Hkv, d, cap
            self.Kc = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, **dev)
            self.Vc = torch.zeros_like(self.Kc)
            self.O = torch.zeros(B, self.N, Hq, d, dtype=torch.float32, **dev)
            self.ws_attn = workspace(tr_verify_attn_workspace_bytes(B, Hq, Hkv, d, cap, tree), device)
            self.scale = d ** -0.5
        self.rope = rope
        if rope is not None:
            if not self.attention or rope.d != d:
                raise ValueError("a rope needs a cache (Hq > 0) with heads of its d")
            self.pos = torch.zeros(B, dtype=torch.int32, **dev)  # tokens before the root, evicted ones too
            self.Q = torch.zeros(B, self.N, Hq, d, dtype=torch.bfloat16, **dev)
            self.Kt = torch.zeros(B, self.N, Hkv, d, dtype=torch.bfloat16, **dev)
            self.Vt = torch.zeros_like(self.Kt)
        self.budget, self.recent, self.scores = budget, recent, None
        if single_token or budget:
            if not self.attention:
                raise ValueError("single-token steps need a cache (Hq > 0)")
            self._init_single_token(dev)
        self._args = make_step_args(tree, self.M, self.tree_tok, self.ids, self.vals, self.acc_len, self.path,
                                    self.committed, self.root, self.L,
                                    logits=torch.empty(1, V, dtype=logits_dtype, **dev) if D == 0 else None,
                                    H=torch.empty(1, max(D, 64), dtype=torch.bfloat16, **dev) if D else None,
                                    Wt=torch.empty(1, max(D, 64), dtype=torch.bfloat16, **dev) if D else None)
        self.ws_step = workspace(tr_step_workspace_bytes(self._args), device)

    def _init_single_token(self, dev):
        """What steps without a draft and eviction need."""
        B, Hq, budget = self.B, self.Hq, self.budget
        if budget:
            if not 0 <= self.recent <= budget:
                raise ValueError("recent must be in [0, budget]")
            # a row that no query has looked at has gathered nothing: scores behind L are always 0
            self.scores = torch.zeros(B, self.Hkv, self.cap, dtype=torch.float32, **dev)
        self.cache = KVCache(self.Kc, self.Vc, self.L, scores=self.scores)
        self.O1 = torch.zeros(B, Hq, self.d, dtype=torch.float32, **dev)
        if self.rope is not None:
            self.Q1 = torch.zeros(B, Hq, self.d, dtype=torch.bfloat16, **dev)
        self.ws_decode = workspace(tr_decode_attn_workspace_bytes(self.cache, Hq, bool(budget)), self.device)
        self.ws_append = workspace(tr_kv_append_workspace_bytes(self.cache), self.device)
        if budget:
            self.ws_evict = workspace(tr_kv_evict_workspace_bytes(self.cache, budget), self.device)
        self.tree1 = Tree((0,), self.K)   # the root alone
        self.ids1 = torch.zeros(B, self.K, dtype=torch.int32, **dev)
        self.path1 = torch.zeros(B, 1, dtype=torch.int32, **dev)
        self.committed1 = torch.zeros(B, 1, dtype=torch.int32, **dev)
        self.ws_topk1 = workspace(tr_topk_workspace_bytes(B, self.V, self.K), self.device)

    def start(self, root, L, M_src=None, mode=TR_INIT_INHERIT, seed=0):
        """Set the roots and cache lengths, initialise M, retrieve the first tree.

        M_src [B, V, K] is copied in as it is; M_src [V, K] is inherited by
        every sequence (tr_init_matrix INHERIT); without M_src, ``mode`` is
        TR_INIT_ZERO or TR_INIT_RANDOM (at ``seed``), or None to keep M as it
        already is."""
        self.root.copy_(torch.as_tensor(root, dtype=torch.int32))
        self.L.copy_(torch.as_tensor(L, dtype=torch.int32))
        if self.rope is not None:
            self.pos.copy_(self.L)
        if self.scores is not None:
            self.scores.zero_()
        if M_src is not None and M_src.dim() == 3:
            self.M.copy_(M_src)
        elif mode is not None:
            tr_init_matrix(self.M, mode, M_src, seed)
        tr_retrieve(self.M, self.tree, self.root, self.tree_tok)

    def rotate(self, Q, K, V):
        """The tree's rows Q [B, N, Hq, d], K, V [B, N, Hkv, d] (views of the projection's
        output), normed and rotated: what verify takes, and finish as Kt and Vt."""
        if self.rope is None:
            raise ValueError("rotate needs a rope")
        tr_qkv_rope(Q, K, V, self.rope, self.pos, self.Q, self.Kt, self.Vt, tree=self.tree)
        return self.Q, self.Kt, self.Vt

    def verify(self, Q, Kt, Vt):
        tr_verify_attn(Q, Kt, Vt, self.Kc, self.Vc, self.L, self.tree, self.O, self.scale, self.ws_attn)
        return self.O

    def finish(self, logits=None, H=None, Wt=None, Kt=None, Vt=None, mode=TR_UPD_ALL, temperature=None, U=None):
        """Everything after the target's forward pass: tr_step, or tr_step_sampled
        at ``temperature`` with the uniforms U [B, N, K+1]."""
        a = make_step_args(self.tree, self.M, self.tree_tok, self.ids, self.vals, self.acc_len, self.path,
                           self.committed, self.root, self.L, logits=logits, H=H, Wt=Wt,
                           Kt=Kt if self.attention else None, Vt=Vt if self.attention else None,
                           Kc=self.Kc if self.attention else None, Vc=self.Vc if self.attention else None,
                           mode=mode, ws=self.ws_step)
        if temperature is None:
            tr_step(a)
        else:
            tr_step_sampled(a, temperature, U)
        if self.rope is not None:
            self.pos.add_(self.acc_len).add_(1)

    def decode(self, Q, Kn, Vn):
        """A step without a draft: appends the root's Kn, Vn [B, Hkv, d] to the cache
        and attends with Q [B, Hq, d] over all its rows (the root's own among
        them); with a budget the rows' weights are gathered.  With a rope Q and Kn are
        normed and rotated first."""
        if self.rope is not None:
            tr_kv_append_rope(Q.unsqueeze(1), Kn.unsqueeze(1), Vn.unsqueeze(1), self.rope, self.cache,
                              self.Q1.unsqueeze(1), self.ws_append, pos=self.pos)
            Q = self.Q1
        else:
            tr_kv_append(Kn.unsqueeze(1), Vn.unsqueeze(1), self.cache, self.ws_append)
        tr_decode_attn(Q, self.cache, self.O1, self.scale, self.ws_decode, accumulate=self.scores is not None)
        return self.O1

    def finish_decode(self, logits, U=None, temperature=None, top_k=None, top_p=None, min_p=None):
        """The end of a step without a draft, from the roots' logits [B, V]: the root's
        row of M becomes its top-K, its first token the next root (committed1).  With the
        uniforms U [B] the next root is drawn by tr_sample instead, with every
        sequence's own rules [B] (refused without U); a row in which nothing can be drawn
        makes the root -1 and sets TR_DEV_BAD_TOKEN.  Tree steps (finish) know one temperature for
        all sequences and no other rule: a loop of both kinds of steps samples from one
        distribution only with that temperature everywhere and no rules here."""
        if U is None and not (temperature is None and top_k is None and top_p is None and min_p is None):
            raise ValueError("temperature, top_k, top_p and min_p need the uniforms U")
        tr_topk(logits, self.K, self.ids1, None, self.ws_topk1, V=self.V)
        tok = self.root.unsqueeze(1)
        tr_update(self.M, self.tree1, tok, self.ids1)
        if U is None:
            tr_accept(self.tree1, tok, self.ids1, self.acc_len, self.path1, self.committed1, self.root)
        else:
            tr_sample(logits, U, self.root, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, V=self.V)
            self.committed1.copy_(tok)   # the root is the drawn token now
            self.acc_len.zero_()
            self.path1.zero_()
        if self.rope is not None:
            self.pos.add_(1)
        tr_retrieve(self.M, self.tree, self.root, self.tree_tok)

    def evict(self):
        """Cuts every sequence longer than the budget down to it: the last ``recent`` rows
        and, for each KV head, those with the most gathered weight."""
        if self.scores is None:
            raise ValueError("evict needs a budget")
        tr_kv_evict(self.cache, self.budget, self.recent, self.ws_evict)
        self.scores[:, :, self.budget:].zero_()   # rows appended there next start from nothing

    def status(self):
        return tr_get_status()
