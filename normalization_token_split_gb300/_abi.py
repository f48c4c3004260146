"""The name of the Python extension.  Its object code holds the layouts of one
interpreter's and one torch's types, so both are part of the name: after another
of either is installed the extension counts as not built, and is not loaded."""
from __future__ import annotations

import importlib.util
import os
import re
import sysconfig


def torch_dir():
    """The installed torch's directory, without importing it; None if there is none."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or spec.origin is None else os.path.dirname(spec.origin)


def torch_version() -> str:
    """The installed torch's version, build tag included ("unknown" if it says none)."""
    try:
        with open(os.path.join(torch_dir() or "", "version.py")) as f:
            said = re.search(r"^__version__\s*(?::[^=]*)?=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        said = None
    return said.group(1) if said else "unknown"


def marshal_name() -> str:
    return f"marshal_nts.{sysconfig.get_config_var('SOABI')}.torch-{torch_version()}.so"
