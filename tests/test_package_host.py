"""The package names its modules."""
import os
import pkgutil

import quantised_linear_layers_gb300 as package


def test_every_public_module_is_named():
    found = {m.name for m in pkgutil.iter_modules(package.__path__) if not m.name.startswith("_")}
    found -= {"build", os.path.splitext("libqlinear.so")[0], "libqlinear_bounds"}
    assert set(package.__all__) == found
    scope = {}
    exec("from quantised_linear_layers_gb300 import *", scope)
    assert set(package.__all__) <= set(scope)
    assert "4-bit" in package.__doc__ and "FP8" in package.__doc__
