"""A small draft model, trained from a larger model's stored top logits and then
used to draft for it: every step but the embedding, the optimiser and the
random numbers runs in the library's kernels.

    python examples/draft_model.py

One block: y = x W, then the block norm (norm of y, gate, residual, norm), then
logits = z H. Training takes rowop_distill's loss and gradient in one call and
goes back through the two products and rowop_block_norm_backward. Serving
samples the draft's tokens (rowop_verify with nothing drafted) and has the
larger model's logits verify them.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import shape_adaptive_tile_gb300 as sat  # noqa: E402

EPS = 1e-6


def _stream():
    return torch.cuda.current_stream().cuda_stream


class Product:
    """C = op(A) op(B) in bf16 with fp32 or bf16 C, one plan for each number of rows."""

    def __init__(self, n, k, c_type, trans_a=False, trans_b=False):
        self.n, self.k, self.c_type, self.trans_a, self.trans_b, self.plans = n, k, c_type, trans_a, trans_b, {}

    def __call__(self, A, B, m, k=None):
        k = k or self.k
        if (m, k) not in self.plans:
            self.plans[m, k] = sat.Plan(m, self.n, k, "bf16", trans_a=self.trans_a, trans_b=self.trans_b, c_type=self.c_type)
        C = torch.empty(m, self.n, device="cuda", dtype=torch.bfloat16 if self.c_type == "bf16" else torch.float32)
        self.plans[m, k].run(A, B, C, 1.0, 0.0, _stream())
        return C


class DraftModel:
    def __init__(self, vocab=4096, width=512, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.vocab, self.width = vocab, width
        self.embedding = torch.randn(vocab, width, device="cuda", generator=g)
        # fp32 weights that the optimiser changes; the products read bf16 copies.
        self.p = {"W": torch.randn(width, width, device="cuda", generator=g) / width ** 0.5,
                  "H": torch.zeros(width, vocab, device="cuda"), "gate": torch.ones(1, width, device="cuda"),
                  "post_gamma": torch.ones(width, device="cuda"), "pre_gamma": torch.ones(width, device="cuda")}
        self.v = {n: torch.zeros_like(t) for n, t in self.p.items()}
        self.xW = Product(width, width, "bf16")
        self.zH = Product(vocab, width, "bf16")
        self.dz = Product(width, vocab, "bf16", trans_b=True)           # dlogits H'
        self.dH = Product(vocab, None, "fp32", trans_a=True)            # z' dlogits
        self.dW = Product(width, None, "fp32", trans_a=True)            # x' dy
        self.copies()

    def copies(self):
        self.W, self.H = self.p["W"].bfloat16(), self.p["H"].bfloat16()

    def _norm_args(self, s, rows):
        return sat.BlockNormArgs(
            rows=rows, width=self.width, block_type="bf16", stream_type="fp32", gate_type="fp32", post_norm="rms", pre_norm="rms",
            post_eps=EPS, pre_eps=EPS, residual_scale=1.0, branch_scale=0.5, x=s["x"], ldx=self.width, y=s["y"], ldy=self.width,
            post_gamma=self.p["post_gamma"], pre_gamma=self.p["pre_gamma"], gate=self.p["gate"], ldg=self.width, rows_per_gate=rows,
            h=s["h"], ldh=self.width, z=s["z"], ldz=self.width, post_stats=s["post_stats"], pre_stats=s["pre_stats"])

    def forward(self, tokens):
        """The logits after each token, and what the backward pass needs."""
        rows = tokens.numel()
        s = {"x": self.embedding[tokens.reshape(-1)]}
        s["x16"] = s["x"].bfloat16()
        s["y"] = self.xW(s["x16"], self.W, rows)
        s["h"], s["z"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        s["post_stats"], s["pre_stats"] = (torch.empty(rows, 2, device="cuda") for _ in range(2))
        sat.check(sat.rowop_block_norm(self._norm_args(s, rows), _stream()))
        s["logits"] = self.zH(s["z"], self.H, rows)
        return s["logits"], s

    def train_step(self, tokens, ids, teacher, rate=0.02, momentum=0.9):
        """One step on rows of a token and the teacher's top logits after it; the rows' mean loss (on the device)."""
        rows, k = ids.shape
        logits, s = self.forward(tokens)
        loss = torch.empty(rows, device="cuda")
        dlogits = torch.empty_like(logits)
        dloss = torch.full((rows,), 1.0 / rows, device="cuda")
        sat.check(sat.rowop_distill(sat.DistillArgs(
            rows=rows, vocab=self.vocab, k=k, logits_type="bf16", teacher_type="fp32", temperature=1.0, logits=logits,
            ldl=self.vocab, ids=ids, ldi=k, teacher=teacher, ldt=k, loss=loss, dloss=dloss, dlogits=dlogits, ldd=self.vocab),
            _stream()))
        dz = self.dz(dlogits, self.H, rows)
        grads = {"H": self.dH(s["z"], dlogits, self.width, rows)}
        args = self._norm_args(s, rows)
        size = sat.rowop_block_norm_workspace(args)
        workspace = torch.empty(size, device="cuda", dtype=torch.uint8)
        dy = torch.empty_like(s["y"])
        for n in ("gate", "post_gamma", "pre_gamma"):
            grads[n] = torch.empty_like(self.p[n])
        sat.check(sat.rowop_block_norm_backward(args, sat.BlockNormGrads(
            dz=dz, lddz=self.width, dy=dy, lddy=self.width, dgate=grads["gate"], lddg=self.width, dpost_gamma=grads["post_gamma"],
            dpre_gamma=grads["pre_gamma"], workspace=workspace, workspace_bytes=size), _stream()))
        grads["W"] = self.dW(s["x16"], dy, self.width, rows)
        for n, t in self.p.items():
            self.v[n].mul_(momentum).add_(grads[n])
            t.add_(self.v[n], alpha=-rate * self.width)
        self.copies()
        return loss.mean()


def verify(target, draft, tokens, generator):
    """(accepted, out) of drafted tokens (batch x drafts), or with draft None and no tokens, samples."""
    batch, drafts = tokens.shape
    vocab = target.shape[-1]
    size = sat.rowop_verify_workspace(batch, drafts, vocab)
    workspace = torch.empty(size, device="cuda", dtype=torch.uint8)
    uniforms = torch.rand(batch, max(drafts, 1), device="cuda", generator=generator)[:, :drafts].contiguous()
    noise = torch.empty(batch, vocab, device="cuda").exponential_(generator=generator).clamp_(min=1e-20)
    accepted = torch.empty(batch, device="cuda", dtype=torch.int32)
    out = torch.empty(batch, drafts + 1, device="cuda", dtype=torch.int32)
    sat.check(sat.rowop_verify(sat.VerifyArgs(
        batch=batch, drafts=drafts, vocab=vocab, logits_type="bf16", temperature=1.0, draft_temperature=1.0, target=target, ldt=vocab,
        draft=draft, ldq=vocab, tokens=tokens if drafts else None, uniforms=uniforms if drafts else None, noise=noise, ldn=vocab,
        accepted=accepted, out=out, workspace=workspace, workspace_bytes=size), _stream()))
    return accepted, out


def serve(model, teacher_logits, first, drafts, generator):
    """Accepted drafts of each sequence: the model drafts from token `first` on, the teacher verifies."""
    batch, said, rows = first.numel(), [first], []
    for _ in range(drafts):
        logits, _ = model.forward(said[-1])
        rows.append(logits)
        _, out = verify(logits, None, torch.empty(batch, 0, device="cuda", dtype=torch.int32), generator)
        said.append(out[:, 0].long())
    draft = torch.stack(rows, 1).contiguous()
    target = teacher_logits(torch.stack(said, 1)).contiguous()
    return verify(target, draft, torch.stack(said[1:], 1).int().contiguous(), generator)[0]


def main(vocab=4096, width=512, batch=1024, k=32, steps=60, drafts=4, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    model = DraftModel(vocab, width)
    # The larger model: the next token's logits are a fixed function of the token.
    inner = torch.randn(vocab, 24, device="cuda", generator=g)
    outer = torch.randn(24, vocab, device="cuda", generator=g)

    def teacher_logits(tokens):
        return (inner[tokens] @ outer).bfloat16()

    first = torch.randint(0, vocab, (256,), device="cuda", generator=g)
    before = serve(model, teacher_logits, first, drafts, g).float().mean()
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch,), device="cuda", generator=g)
        top, ids = teacher_logits(tokens).float().topk(k, dim=-1)  # what would have been stored
        losses.append(model.train_step(tokens, ids.int().contiguous(), top.contiguous()))
    after = serve(model, teacher_logits, first, drafts, g).float().mean()
    losses = torch.stack(losses).tolist()
    print(f"distillation loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps; "
          f"accepted of {drafts} drafted tokens {before:.2f} -> {after:.2f}")
    return losses, float(before), float(after)


if __name__ == "__main__":
    main()
