"""MI355X-native per-matrix Muon update (HIP kernels for gfx950 behind a C-ABI library).

``binding`` (loaded on first use) marshals arguments into ``libmuon_amd.so``; every step
of the update runs in the library's HIP kernels. The operators a training step runs before
the update: ``layers`` (gated feed-forward block), ``mixers`` (linear attention with decay),
``experts`` (tokens sorted by expert and back), ``dropout`` and ``losses`` (vocabulary losses).
``workloads`` holds the seeded synthetic inputs.
"""

import importlib

__all__ = ["binding", "dropout", "experts", "layers", "losses", "mixers", "workloads"]


def __getattr__(name):
    if name in __all__:
        return importlib.import_module(f"{__name__}.{name}")
    raise AttributeError(name)
