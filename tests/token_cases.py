"""Sizes of the cross entropy over a vocabulary that lead to its large tiles, to several
pieces of the vocabulary and to several passes over the tokens, and what its plan makes of
them: `tests/test_token_loss_plan_host.py` holds the plan to it, `tests/test_gpu_token_edges.py`
the results."""

# name: (T, V, C, type, share of tokens without a target, what the plan has to say)
LOSS_PLANS = {
    "wide logits": (3900, 4090, 264, "bf16", 0.01,
                    {"forward": 256, "logits": 256, "pieces": 1}),
    "wide g_x": (7100, 300, 2056, "bf16", 0.0, {"singles": 256, "pieces": 1}),
    "wide g_W": (500, 3000, 4104, "bf16", 0.05, {"weights": 256, "pieces": 1}),
    "pieces": (65536, 5393, 200, "bf16", 0.998,
               {"forward": 256, "logits": 256, "singles": 256, "weights": 128, "pieces": 6,
                "piece": 1024, "last": 273}),
    "pieces and passes": (66100, 5393, 200, "bf16", 0.998,
                          {"tokens": 65536, "logits": 256, "pieces": 6, "last": 273}),
    "pieces f32": (65536, 5393, 64, "f32", 0.998,
                   {"forward": 128, "logits": 128, "singles": 64, "weights": 64, "pieces": 4,
                    "piece": 1536, "last": 785}),
    "wide logits f32": (6140, 6130, 8, "f32", 0.01, {"forward": 128, "logits": 128}),
    "wide g_x f32": (36860, 16, 1024, "f32", 0.97, {"singles": 128}),
    "wide g_W f32": (40, 36860, 1024, "f32", 0.0, {"weights": 128}),
    "small tiles": (300, 1301, 128, "bf16", 0.2,
                    {"forward": 128, "logits": 128, "singles": 128, "weights": 128}),
    "small tiles f32": (300, 1301, 128, "f32", 0.2,
                        {"forward": 64, "logits": 64, "singles": 64, "weights": 64}),
}
