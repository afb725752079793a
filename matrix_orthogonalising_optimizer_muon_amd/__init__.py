"""MI355X-native per-matrix Muon update (HIP kernels for gfx950 behind a C-ABI library).

``binding`` (loaded on first use) marshals arguments into ``libmuon_amd.so``; every step
of the update runs in the library's HIP kernels. ``layers`` and ``losses`` are the operators a
training step runs before the update (gated feed-forward block, vocabulary losses).
``workloads`` holds the seeded synthetic inputs.
"""

import importlib

__all__ = ["binding", "layers", "losses", "workloads"]


def __getattr__(name):
    if name in __all__:
        return importlib.import_module(f"{__name__}.{name}")
    raise AttributeError(name)
